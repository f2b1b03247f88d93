"""The pages' two-chunk layer step on one GPU ("TokenWeave: Efficient
Compute-Communication Overlap for Distributed LLM Inference", gist.science
summary, "Der intelligente Split" and "Der Fused Kernel").

A row-parallel linear layer leaves its output in partial 0 (the other
partials stand for the other ranks' outputs).  The batch is cut into two token
chunks A and B: the GEMM of chunk A runs first; then the GEMM of chunk B runs
on its stream while the fused reduce + residual add + RMSNorm of chunk A runs
beside it on a second stream, held to a few SMs; the fused step of chunk B
follows its GEMM with the whole GPU.  Events order each fused step after the
GEMM that writes its rows.

The GEMM of the bf16 steps is a plain library GEMM (``torch.matmul``, cuBLAS):
the compute the pages overlap with, not part of the fused path.  Every step of
the fused path runs in libtw.so.  The 8-bit step
(:func:`two_chunk_layer_step_q8`) runs its product there too, and hands the
normalised rows on in 8 bits.
"""
import torch

from . import tw


def two_chunk_layer_step(x, wmat, partials, residual, weight, out, residual_out, eps,
                         budget, gemm_stream, fused_stream, t_split=None):
    """Enqueue one two-chunk layer step.

    ``x`` [T, K] and ``wmat`` [K, H] give partial 0 = x @ wmat ([T, H], written
    chunk by chunk); chunk A is tokens [0, t_split) (default T // 2), fused on
    ``fused_stream`` under a budget of ``budget`` SMs beside the GEMM of chunk
    B; chunk B is fused with the whole GPU once its GEMM is done.  On return
    ``gemm_stream`` is ordered after the whole step."""
    T = residual.shape[0]
    split = T // 2 if t_split is None else t_split
    done_a, done_b = torch.cuda.Event(), torch.cuda.Event()
    with torch.cuda.stream(gemm_stream):
        torch.matmul(x[:split], wmat, out=partials[0][:split])
        done_a.record(gemm_stream)
        torch.matmul(x[split:], wmat, out=partials[0][split:])
        done_b.record(gemm_stream)
    fused_stream.wait_event(done_a)
    tw.tw_fused_reduce_add_rmsnorm(partials, residual, weight, out, residual_out, eps, 0, split,
                                   max_sms=budget, stream=fused_stream)
    fused_stream.wait_event(done_b)
    tw.tw_fused_reduce_add_rmsnorm(partials, residual, weight, out, residual_out, eps, split, T,
                                   stream=fused_stream)
    gemm_stream.wait_stream(fused_stream)


def sequential_layer_step(x, wmat, partials, residual, weight, out, residual_out, eps, stream):
    """The same layer without the split: the whole GEMM, then the fused step
    with the whole GPU, on one stream."""
    with torch.cuda.stream(stream):
        torch.matmul(x, wmat, out=partials[0])
    tw.tw_fused_reduce_add_rmsnorm(partials, residual, weight, out, residual_out, eps,
                                   stream=stream)


def two_chunk_layer_step_q8(x, x_scale, w, w_scale, partials, residual, weight, out, out_scale,
                            residual_out, eps, budget, gemm_stream, fused_stream, t_split=None):
    """The two-chunk step of a layer served in 8 bits.

    ``x`` [T, K] with ``x_scale`` [T] and ``w`` [H, K] with ``w_scale`` [H]
    (int8 or float8_e4m3fn) give partial 0 = the scaled product, chunk by chunk;
    the fused steps write ``out`` in 8 bits with ``out_scale``, the next linear
    layer's input.  The product of chunk B leaves ``budget`` SMs to the fused
    step of chunk A beside it.  On return ``gemm_stream`` is ordered after the
    whole step.

    On one GPU this pays only where the product of a chunk lasts as long as the
    fused step of the other on ``budget`` SMs: with 8 partials of 16384 x 8192
    and K = 8192, 1500 us (int8, 32 SMs) against 1514 for the product and the
    fused step called in turn on one stream, and 994 against 999 in e4m3 (48
    SMs); with K = 1024 or 2048 tokens the calls in turn are faster (2048 x 8192
    over K = 8192: 203 us against 221 in int8, 140 against 149 in e4m3)."""
    T = residual.shape[0]
    split = T // 2 if t_split is None else t_split
    sms = torch.cuda.get_device_properties(residual.device).multi_processor_count
    done_a, done_b = torch.cuda.Event(), torch.cuda.Event()
    tw.tw_gemm_q8(x, x_scale, w, w_scale, partials[0], 0, split, stream=gemm_stream)
    done_a.record(gemm_stream)
    tw.tw_gemm_q8(x, x_scale, w, w_scale, partials[0], split, T, max_sms=max(1, sms - budget),
                  stream=gemm_stream)
    done_b.record(gemm_stream)
    args = (partials, residual, weight, out, out_scale, residual_out, eps)
    fused_stream.wait_event(done_a)
    tw.tw_fused_reduce_add_rmsnorm_q8(*args, 0, split, max_sms=budget, stream=fused_stream)
    fused_stream.wait_event(done_b)
    tw.tw_fused_reduce_add_rmsnorm_q8(*args, split, T, stream=fused_stream)
    gemm_stream.wait_stream(fused_stream)
