"""MI355X all-reduce family: one-shot, two-shot and ring all-reduce,
reduce-scatter and all-gather over N simulated rank buffers on one GPU, with
Simple, LL and LL128 transports, and the operators of a tensor-parallel layer
whose partial sums they add: a gated feed-forward block and a linear cross
entropy over a split vocabulary, with their gradients, query and key norms with
the position rotation, and attention over an 8-bit key/value cache.  The work
runs in hand-written HIP kernels (libar.so, C ABI in include/ar.h); ``binding``
marshals arguments to it."""

from .binding import (ACTS, ALGOS, DTYPES, OPS, PROTOS, ARError, Comm, KVCache, allreduce_noalloc,  # noqa: F401
                      cache_attention, cache_read, cache_write, gated_ffn, gated_ffn_backward, library,
                      linear_cross_entropy, linear_cross_entropy_backward, plan_bytes, qk_norm_rope,
                      qk_norm_rope_backward, select, stream_ceiling, vocab_shards)
