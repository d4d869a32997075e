"""GB300-native AdamW optimizer step (pure-bf16 Kahan and fp32-master mixed
modes) behind a small C ABI; see ``adamw_sm`` for the binding, ``optim`` for
the ``torch.optim`` front ends and the clip over all their groups, and
``losses`` for the fine-tuning losses that feed them."""
