"""GB300-native AdamW optimizer step (pure-bf16 Kahan and fp32-master mixed
modes) behind a small C ABI; see ``adamw_sm`` for the binding, ``optim`` for
the ``torch.optim`` front ends (Muon among them) and the clip over all their
groups, ``losses`` for the fine-tuning losses that feed them, and ``matrix`` for
orthogonalisation and products grouped by expert."""
