"""MI355X all-reduce family: one-shot, two-shot and ring all-reduce,
reduce-scatter and all-gather over N simulated rank buffers on one GPU, with
Simple, LL and LL128 transports, and the operators of a tensor-parallel layer
whose partial sums they add: a gated feed-forward block and a linear cross
entropy over a split vocabulary, with their gradients.  The work runs in hand-written HIP kernels
(libar.so, C ABI in include/ar.h); ``binding`` marshals arguments to it."""

from .binding import (ACTS, ALGOS, DTYPES, OPS, PROTOS, ARError, Comm, allreduce_noalloc,  # noqa: F401
                      gated_ffn, gated_ffn_backward, library, linear_cross_entropy,
                      linear_cross_entropy_backward, plan_bytes, select, stream_ceiling, vocab_shards)
