"""zero_sharded_mixed_flat_gb300: the sharded mixed-precision optimizer step
(ZeRO stage two over a flat parameter vector) as hand-written CUDA for GB300.

The compute lives in the C-ABI library ``libzg.so`` (sources in ``csrc/``,
declarations in ``include/zg.h``). ``binding`` is a thin ctypes layer over it
that takes torch tensors for device memory and streams. ``synth`` draws the
seeded synthetic inputs and ``accounting`` holds the byte formulas.

Beside the step the library has training operators that give it its gradients:
the gated linear recurrence over time (``binding.GatedScan``), the selection of
a teacher's top logits (``binding.topk_logits``) and the distillation loss on
them with its gradient (``binding.distill_loss``, ``distill_grad``,
``distill_loss_grad``); the token embedding (``embed``, ``embed_grad``), the norms
around a block with its gate and residual scale (``block_norm``,
``block_norm_grad``), the clipped policy loss with its gradient (``token_logp``,
``policy_loss``, ``policy_grad``, ``policy_loss_grad``) and the clipping of many
gradients into the flat one (``GradClip``). Their sources are in ``csrc/ops/``.

Importing this package loads nothing; the library is loaded on first use of
``binding`` and the import fails loudly if it has not been built.
"""

__all__ = ["binding", "synth", "accounting"]
