// tw_rows.cu -- the rows kernel's launch plan, and its instantiations with
// outputs of the input dtype (tw_rows_q8.cu holds those with 8-bit outputs).
#include "tw_rows.cuh"

namespace tw {
namespace {

void* rows_kernel_for(int dtype, int nv, int unit, int mode, bool q8) {
    return q8 ? rows_q8_entry(dtype, nv, unit, mode) : rows_entry<false>(dtype, nv, unit, mode);
}

void* rows2_kernel_for(int dtype, int nv, int unit, bool q8) {
    return q8 ? rows2_q8_entry(dtype, nv, unit) : rows2_entry<false>(dtype, nv, unit);
}

int rows_vectors_per_thread(int64_t row_bytes, int threads = kRowsThreads) {
    return static_cast<int>((row_bytes / 16 + threads - 1) / threads);
}

// Tokens of the busiest CTA when `tokens` tokens are cut into units of u
// (the last one ragged) dealt round robin to min(units, sms) CTAs.
int64_t busiest_cta_tokens(int64_t tokens, int64_t u, int64_t sms) {
    const int64_t units = (tokens + u - 1) / u;
    const int64_t grid = units < sms ? units : sms;
    const int64_t full = (units + grid - 1) / grid;  // units of the busiest CTAs
    const int64_t r = units % grid;
    const int64_t n_busiest = r == 0 ? grid : r;
    if (n_busiest >= 2) return full * u;  // one of them holds whole units only
    // The only busiest CTA (CTA 0) also holds the ragged last unit.
    const int64_t last = tokens - (units - 1) * u;
    return full * u - (u - last);
}

}  // namespace

size_t rows_smem_bytes(size_t stage_bytes, int stages) {
    return static_cast<size_t>(kRingOff) + static_cast<size_t>(stages) * stage_bytes;
}

int rows_unit_tokens(const Params& p, int64_t tokens, int64_t sms) {
    // Units of several tokens only where one copy per row would be small and
    // the unit does not lengthen the busiest CTA's share of the range: the
    // largest U with U * row <= kUnitCopyBytes, U * vectors per thread within
    // the register budget, and the busiest CTA's tokens no more than with
    // one token per unit.  Readiness flags and the column-split mode take
    // one token per unit.
    if (p.ready || p.colsplit || tokens < 1 || sms < 1) return 1;
    const int nv = rows_vectors_per_thread(p.row_bytes);
    const int64_t share1 = busiest_cta_tokens(tokens, 1, sms);
    for (int u = kRowsMaxUnit; u > 1; u /= 2) {
        if (u * p.row_bytes > kUnitCopyBytes || u * nv > kRowsMaxVecs) continue;
        if (busiest_cta_tokens(tokens, u, sms) <= share1) return u;
    }
    return 1;
}

size_t rows_plan(Params& p, int smem_optin) {
    // Whole row groups of one unit per stage: the whole unit if its R groups
    // fit kStageTargetBytes, else the unit's groups split evenly over the
    // fewest stages that fit (never more than R groups).  As many stages as
    // fit the shared memory.  p.unit_tokens must be set.
    const int64_t rows = p.colsplit ? 2 : p.n_parts + 1;
    const int64_t group = p.unit_tokens * p.row_bytes;
    const int64_t parts = (rows * group + kStageTargetBytes - 1) / kStageTargetBytes;
    int64_t per_stage = (rows + parts - 1) / parts;
    if (per_stage * group > kStageTargetBytes) per_stage = kStageTargetBytes / group;
    if (per_stage < 1) per_stage = 1;
    const size_t stage = static_cast<size_t>(per_stage * group);
    int stages = static_cast<int>((static_cast<size_t>(smem_optin) - rows_smem_bytes(0, 0)) / stage);
    if (stages > kMaxStages) stages = kMaxStages;
    if (stages < kMinStages) return 0;
    // Producer warps: the largest power of two up to kRowsMaxProducers that
    // the ring holds; the ring is cut to a multiple of it, so each producer
    // owns the same stages for the whole launch.
    static_assert((kRowsMaxProducers & (kRowsMaxProducers - 1)) == 0,
                  "producer count must be a power of two");
    int producers = kRowsMaxProducers;
    while (producers > 1 && producers > stages) producers /= 2;
    stages -= stages % producers;
    p.rows_per_stage = static_cast<int>(per_stage);
    p.stages = stages;
    p.producers = producers;
    const size_t smem = rows_smem_bytes(stage, stages);
    return smem < static_cast<size_t>(kExclusiveSmemBytes) ? kExclusiveSmemBytes : smem;
}

bool rows_two_pipes_fit(const Params& p, bool budgeted) {
    // Two pipelines: the fixed schedule, at least two ring stages each, and a
    // unit's x in registers with 256 threads per group.  Under an SM budget
    // they always pay (8 SMs: 291 -> 266 us on N = 8, H = 8192; 190 -> 156
    // us on N = 2, H = 4096).  With the whole GPU only when a pipeline's half
    // of the ring holds a whole unit (N = 2: 14.3 -> 13.6 us); otherwise
    // each pipeline would wait for its own first stage to be read before it
    // could fetch a unit's last one (N = 8: 28.2 -> 28.6 us).
    const int nv2 = rows_vectors_per_thread(p.row_bytes, kRowsThreads / 2);
    if (p.ready || p.work || p.stages < 4 || p.unit_tokens * nv2 > kRowsMaxVecs ||
        rows2_kernel_for(TW_BF16, nv2, p.unit_tokens, false) == nullptr)
        return false;
    const int rows = p.colsplit ? 2 : p.n_parts + 1;
    const int stages_per_unit = (rows + p.rows_per_stage - 1) / p.rows_per_stage;
    return budgeted || stages_per_unit <= p.stages / 2;
}

int rows_set_smem_limit(int smem_optin, bool q8) {
    for (int dt = 0; dt < 2; ++dt)
        for (int nv = 1; nv <= kRowsMaxVecs; ++nv)
            for (int unit = 1; unit <= kRowsMaxUnit; unit *= 2) {
                void* fns[] = {rows_kernel_for(dt, nv, unit, kFixed, q8),
                               rows_kernel_for(dt, nv, unit, kClaim, q8),
                               rows_kernel_for(dt, nv, unit, kFlags, q8),
                               rows2_kernel_for(dt, nv, unit, q8)};
                for (void* fn : fns) {
                    if (!fn) continue;
                    cudaError_t e = cudaFuncSetAttribute(
                        fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_optin);
                    if (e != cudaSuccess) return static_cast<int>(e);
                }
            }
    return 0;
}

int launch_rows(const Params& p, int dtype, int grid, size_t smem_bytes, bool pdl,
                void* stream) {
    void* fn;
    if (p.pipes == 2) {
        fn = rows2_kernel_for(dtype, rows_vectors_per_thread(p.row_bytes, kRowsThreads / 2),
                              p.unit_tokens, p.q8 != 0);
    } else {
        const int mode = p.ready ? kFlags : p.work ? kClaim : kFixed;
        fn = rows_kernel_for(dtype, rows_vectors_per_thread(p.row_bytes), p.unit_tokens, mode,
                             p.q8 != 0);
    }
    if (!fn) return static_cast<int>(cudaErrorInvalidValue);
    return launch_with_pdl(fn, p, grid, kRowsBlock, smem_bytes, pdl, stream);
}

}  // namespace tw
