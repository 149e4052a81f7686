// HIP kernels of the ZeRO shard step for gfx950 (CDNA4, wave64).
//
// The step is a pure stream: every shard element is read once from each of
// the N gradient partials and from the fp32 master, m and v, and written
// once to master, m, v and the bf16 parameter slot.  Nothing is reused, so
// the bound is HBM bandwidth: (2N + 26) bytes per element with bf16
// partials, (4N + 26) with fp32 partials.  There is no contraction here,
// so no MFMA; the kernels are built around 16-byte per-lane accesses that
// a wave turns into fully coalesced 1 KiB requests.
//
// Work split: one workgroup (a single wave of 64 lanes) per chunk of the
// chunk table (a workgroup loops over chunks when the table is longer than
// the grid cap).  A lane handles a group of VEC consecutive elements (8
// with bf16 partials: one 16-byte load per partial; 4 with fp32 partials),
// strided by the wave width; the default 2048-element chunk is four groups
// per lane.  Groups sit on the shard's VEC-element grid, so all
// partial and state loads are 16-byte aligned; a chunk that starts or ends
// off the grid handles its first or last group element by element.
//
// Arithmetic follows the fixed evaluation order in include/zero_shard.h:
// double sums in rank order, IEEE double AdamW without contraction (the
// library is built with -ffp-contract=off), one rounding per stored value.

#include "zero_device.h"

namespace zs {

template <zero_dtype G, int NC>
__global__ __launch_bounds__(kStepBlock) __attribute__((amdgpu_waves_per_eu(1, kKahanWaves)))
void shard_step_kahan_kernel(StepArgs a)
{
    for (int64_t ci = blockIdx.x; ci < a.n_chunks; ci += gridDim.x)
        step_chunk_kahan<G, NC>(a, chunk_at(a.chunks, ci), a.k);
}

template <zero_dtype G, int NC, bool SMALL>
__global__ __launch_bounds__(kStepBlock) __attribute__((amdgpu_waves_per_eu(1, kM16Waves<G, NC, SMALL>)))
void shard_step_m16_kernel(StepArgs a)
{
    for (int64_t ci = blockIdx.x; ci < a.n_chunks; ci += gridDim.x)
        step_chunk_m16<G, NC, SMALL>(a, chunk_at(a.chunks, ci), a.k);
}

// In every chunk-table kernel a workgroup (one wave) takes chunks
// blockIdx.x, blockIdx.x + gridDim.x, ...: the grid is capped so that
// work-items stay below 2^32 however long the table is.
//
// On large launches the 16-byte step keeps at most one wave per SIMD
// (waves_per_eu): with fewer concurrent streams the HBM sustains more of its
// peak on this mixed read/write stream.  Measured on MI355X with occupancy
// capped exactly by LDS reservations, one process, same buffers: 4 resident
// waves per CU beat 3 and 5-8 (7B shard 0.721 against 0.669 and
// 0.648-0.705; 70B 0.761 against 0.702 and 0.747-0.751).  Each wave still
// keeps its group's 14 (N = 8) to 22 (N = 16) 16-byte loads in flight.
//
// KC (extended step only): -1 flat rank order, 0 two-level with the group
// size at run time, > 0 two-level with that group size.
//
// W: resident waves per SIMD.  A launch of at most ZERO_SMALL_LAUNCH_CHUNKS
// chunks (a small shard, or one gradient bucket) runs two: with few
// workgroups per CU the launch's ramp and tail weigh more than the
// read/write mix.  Measured on MI355X, N = 8 bf16, chunks of 2048, one
// process, each launch on the next of enough buffer sets to keep the
// working set (over 2 GB) out of the 256 MB last-level cache, one wave
// against two: 2M-element shards 0.45 / 0.44-0.45, 4M 0.49-0.50 /
// 0.51-0.52, 8M 0.58 / 0.57-0.58, 16M 0.62-0.64 / 0.60, 32M 0.68-0.70 /
// 0.67, 64M 0.70-0.71 / 0.68; 7B gradient buckets of 4M params (2048
// chunks) 0.547 / 0.568, of 16M (8192 chunks) 0.662 / 0.652.  (Re-stepping
// one buffer set instead favours two waves up to 16M elements, 0.79 against
// 0.71 there, because part of the set then stays in that cache.)
//
// The allocation behind one wave per SIMD: with amdgpu_waves_per_eu(1, 1)
// the compiler declares 257 registers (.amdhsa_next_free_vgpr; 114 of them
// used), and 257 rounded to gfx950's granule of 8 fills more than half of
// a SIMD's 512, so only one such wave fits.  The two-wave instance declares
// 169 (176 allocated, two fit).  rocprofv3 reports the 257 as "132" (it
// counts granules of 4).
//
// The extended step picks its divisor path once per chunk, with a uniform
// branch around the whole chunk, instead of per element inside the unrolled
// loop.  On MI355X, bitwise equal, same buffers: 7B 0.696 -> 0.707 (K = 4),
// 0.648 -> 0.663 (K = 2, fold at run time), 0.697 -> 0.703 (three
// micro-batches, so divided); 70B 0.730 -> 0.740 (K = 8).
template <zero_dtype G, int NC, bool EXT, int KC = -1, int W = 1>
__global__ __launch_bounds__(kStepBlock) __attribute__((amdgpu_waves_per_eu(1, W)))
void shard_step_kernel(StepArgs a)
{
    for (int64_t ci = blockIdx.x; ci < a.n_chunks; ci += gridDim.x) {
        if constexpr (EXT) {
            if (a.red.pow2)
                step_chunk<G, NC, EXT, KC, 1>(a, chunk_at(a.chunks, ci), a.k);
            else
                step_chunk<G, NC, EXT, KC, 2>(a, chunk_at(a.chunks, ci), a.k);
        } else {
            step_chunk<G, NC, EXT, KC>(a, chunk_at(a.chunks, ci), a.k);
        }
    }
}

// The fused steps with their constants in device memory: entry
// *a.sched_index of the table a.sched (formed on the host, as the
// launch-argument constants are).  A graph that captures this launch applies
// whichever step the index names when it replays.  An index outside the
// table leaves everything untouched.  L: the state layout (0: fp32 master,
// m, v; 1: fp32 master, bf16 m, v; 2: pure bf16 with compensation), each
// with the occupancy of its launch-argument kernel (SMALL: chosen per
// launch as for those kernels).
template <int L, zero_dtype G, int NC, bool SMALL>
constexpr int kSchedWaves = L == 0 ? (SMALL ? 2 : 1)
                                   : (L == 1 ? kM16Waves<G, NC, SMALL> : kKahanWaves);

template <int L, zero_dtype G, int NC, bool SMALL>
__global__ __launch_bounds__(kStepBlock) __attribute__((amdgpu_waves_per_eu(1, kSchedWaves<L, G, NC, SMALL>)))
void shard_step_sched_kernel(StepArgs a)
{
    const int64_t t = *(const_i64 *)a.sched_index;
    if (t < 0 || t >= a.n_sched)
        return;
    const const_f64 *e = (const const_f64 *)(a.sched + t);
    StepScalars k;
    k.b1 = e[0]; k.c1 = e[1]; k.b2 = e[2]; k.c2 = e[3]; k.bc1 = e[4]; k.bc2 = e[5];
    k.eps = e[6]; k.lr = e[7]; k.dec = e[8]; k.wd = e[9];
    for (int64_t ci = blockIdx.x; ci < a.n_chunks; ci += gridDim.x) {
        if constexpr (L == 0)
            step_chunk<G, NC, false, -1>(a, chunk_at(a.chunks, ci), k);
        else if constexpr (L == 1)
            step_chunk_m16<G, NC, SMALL>(a, chunk_at(a.chunks, ci), k);
        else
            step_chunk_kahan<G, NC>(a, chunk_at(a.chunks, ci), k);
    }
}

// *index += 1 when 0 <= *index < n (one lane, a vector store).
__global__ __launch_bounds__(64) void step_index_advance_kernel(int64_t *index, int64_t n)
{
    if (threadIdx.x == 0) {
        const int64_t t = index[0];
        if (t >= 0 && t < n)
            index[0] = t + 1;
    }
}

// ---------------------------------------------------------------- unfused

template <zero_dtype G, int NC>
__global__ __launch_bounds__(kBlock) void reduce_kernel(ReduceArgs a)
{
    constexpr int VEC = Grad<G>::VEC;
    const int n = NC > 0 ? NC : a.red.n_ranks;
    const int64_t groups = a.n / VEC;
    for (int64_t g = (int64_t)blockIdx.x * kBlock + threadIdx.x; g < groups;
         g += (int64_t)gridDim.x * kBlock) {
        const int64_t i0 = g * VEC;
        double s[VEC];
        group_sum<G, NC>(s, a.parts, n, i0);
        F32x<VEC> out;
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            out[j] = finish_reduce<NC>(s[j], a.red);
        out.store(a.out + i0);
    }
    if (blockIdx.x == 0) {
        const int64_t i = groups * VEC + threadIdx.x;
        if (i < a.n)
            a.out[i] = finish_reduce<NC>(elem_sum<G>(a.parts, n, i), a.red);
    }
}

// One non-final micro-batch: acc = fp32((reset ? 0 : acc) + two-level sum).
// Launched like the step kernel: one wave per workgroup, at most one wave
// per SIMD; workgroup b walks spans b, b + gridDim.x, ... of kAccSpan
// consecutive elements.
constexpr int64_t kAccSpan = 2048;

template <zero_dtype G, int NC, int KC>
__global__ __launch_bounds__(kStepBlock) __attribute__((amdgpu_waves_per_eu(1, 1)))
void accumulate_kernel(AccArgs a)
{
    constexpr int VEC = Grad<G>::VEC;
    constexpr int64_t GPS = kAccSpan / VEC;   // groups per span
    const int n = NC > 0 ? NC : a.red.n_ranks;
    const int64_t groups = a.n / VEC;
    for (int64_t sp = blockIdx.x; sp * GPS < groups; sp += gridDim.x) {
        const int64_t gend = (sp + 1) * GPS < groups ? (sp + 1) * GPS : groups;
        for (int64_t g = sp * GPS + threadIdx.x; g < gend; g += kStepBlock) {
            const int64_t i0 = g * VEC;
            F32x<VEC> acc;
            if (!a.reset)
                acc.load(a.acc + i0);
            double s[VEC];
            if constexpr (KC < 0)
                group_sum<G, NC>(s, a.parts, n, i0);
            else
                group_sum_two_level<G, NC, KC>(s, a.parts, n, a.red.group, i0);
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                acc[j] = a.reset ? (float)s[j] : (float)((double)acc[j] + s[j]);
            acc.store(a.acc + i0);
        }
    }
    if (blockIdx.x == 0) {
        const int64_t i = groups * VEC + threadIdx.x;   // the last n % VEC elements
        if (i < a.n) {
            const double e = elem_sum_two_level<G>(a.parts, n, a.red.group, i);
            a.acc[i] = a.reset ? (float)e : (float)((double)a.acc[i] + e);
        }
    }
}

__global__ __launch_bounds__(kBlock) void adamw_kernel(AdamArgs a)
{
    const int64_t groups = a.n / 4;
    for (int64_t g = (int64_t)blockIdx.x * kBlock + threadIdx.x; g < groups;
         g += (int64_t)gridDim.x * kBlock) {
        const int64_t i0 = g * 4;
        F32x<4> gr, th, m, v;
        gr.load(a.g + i0);
        th.load(a.master + i0);
        m.load(a.m + i0);
        v.load(a.v + i0);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            adamw(gr[j], th[j], m[j], v[j], a.k);
        th.store(a.master + i0);
        m.store(a.m + i0);
        v.store(a.v + i0);
    }
    if (blockIdx.x == 0) {
        const int64_t i = groups * 4 + threadIdx.x;
        if (i < a.n) {
            float th = a.master[i], m = a.m[i], v = a.v[i];
            adamw(a.g[i], th, m, v, a.k);
            a.master[i] = th;
            a.m[i] = m;
            a.v[i] = v;
        }
    }
}

__device__ __forceinline__ void gather_chunk(const GatherArgs &a, const zero_chunk &c)
{
    constexpr int VEC = 8;
    if (c.len <= 0 || c.shard_off < 0 || c.shard_off > a.shard_len - c.len)
        return;
    const int64_t lo = c.shard_off, hi = c.shard_off + c.len;
    const int64_t g0 = lo / VEC, g1 = (hi + VEC - 1) / VEC;
    const bool vec_ok = (((uintptr_t)c.dst - (uintptr_t)(2 * (lo - g0 * VEC))) % (2 * VEC)) == 0;
    ParamStore<VEC> ps(c.dst, lo, hi, vec_ok);
    for (int64_t g = g0 + threadIdx.x; g < g1; g += kStepBlock) {
        const int64_t i0 = g * VEC;
        uint16_t *d = c.dst + (i0 - lo);
        if (i0 >= lo && i0 + VEC <= hi) {
            F32x<VEC> th;
            th.load(a.master + i0);
            uint32_t h[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                h[j] = to_bf16(th[j]);
            ps.put(i0, h);
        } else {
            for (int j = 0; j < VEC; ++j) {
                const int64_t i = i0 + j;
                if (i >= lo && i < hi)
                    d[j] = (uint16_t)to_bf16(a.master[i]);
            }
        }
    }
}

__global__ __launch_bounds__(kStepBlock) __attribute__((amdgpu_waves_per_eu(1, 1)))
void gather_kernel(GatherArgs a)
{
    for (int64_t ci = blockIdx.x; ci < a.n_chunks; ci += gridDim.x)
        gather_chunk(a, chunk_at(a.chunks, ci));
}

// ---------------------------------------------------------------- launchers

static int grid_for(int64_t items)
{
    // Enough workgroups to fill 256 CUs many times over; the kernels stride.
    int64_t blocks = (items + kBlock - 1) / kBlock;
    if (blocks > 256 * 64)
        blocks = 256 * 64;
    return blocks < 1 ? 1 : (int)blocks;
}

template <zero_dtype G, int W>
static hipError_t step_dispatch(const StepArgs &a, hipStream_t s)
{
    dim3 grid(chunk_grid(a.n_chunks)), block(kStepBlock);
    switch (a.red.n_ranks) {
    case 1: hipLaunchKernelGGL((shard_step_kernel<G, 1, false, -1, W>), grid, block, 0, s, a); break;
    case 2: hipLaunchKernelGGL((shard_step_kernel<G, 2, false, -1, W>), grid, block, 0, s, a); break;
    case 4: hipLaunchKernelGGL((shard_step_kernel<G, 4, false, -1, W>), grid, block, 0, s, a); break;
    case 8: hipLaunchKernelGGL((shard_step_kernel<G, 8, false, -1, W>), grid, block, 0, s, a); break;
    case 16: hipLaunchKernelGGL((shard_step_kernel<G, 16, false, -1, W>), grid, block, 0, s, a); break;
    case 32: hipLaunchKernelGGL((shard_step_kernel<G, 32, false, -1, W>), grid, block, 0, s, a); break;
    case 64: hipLaunchKernelGGL((shard_step_kernel<G, 64, false, -1, W>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((shard_step_kernel<G, 0, false, -1, W>), grid, block, 0, s, a); break;
    }
    return hipGetLastError();
}

hipError_t launch_step(const StepArgs &a, zero_dtype gdt, hipStream_t s)
{
    const bool small = a.n_chunks <= ZERO_SMALL_LAUNCH_CHUNKS;
    if (gdt == ZERO_BF16)
        return small ? step_dispatch<ZERO_BF16, 2>(a, s) : step_dispatch<ZERO_BF16, 1>(a, s);
    return small ? step_dispatch<ZERO_FP32, 2>(a, s) : step_dispatch<ZERO_FP32, 1>(a, s);
}

template <int L, zero_dtype G, bool SMALL>
static hipError_t step_sched_dispatch(const StepArgs &a, hipStream_t s)
{
    dim3 grid(chunk_grid(a.n_chunks)), block(kStepBlock);
    switch (a.red.n_ranks) {
    case 1: hipLaunchKernelGGL((shard_step_sched_kernel<L, G, 1, SMALL>), grid, block, 0, s, a); break;
    case 2: hipLaunchKernelGGL((shard_step_sched_kernel<L, G, 2, SMALL>), grid, block, 0, s, a); break;
    case 4: hipLaunchKernelGGL((shard_step_sched_kernel<L, G, 4, SMALL>), grid, block, 0, s, a); break;
    case 8: hipLaunchKernelGGL((shard_step_sched_kernel<L, G, 8, SMALL>), grid, block, 0, s, a); break;
    case 16: hipLaunchKernelGGL((shard_step_sched_kernel<L, G, 16, SMALL>), grid, block, 0, s, a); break;
    case 32: hipLaunchKernelGGL((shard_step_sched_kernel<L, G, 32, SMALL>), grid, block, 0, s, a); break;
    case 64: hipLaunchKernelGGL((shard_step_sched_kernel<L, G, 64, SMALL>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((shard_step_sched_kernel<L, G, 0, SMALL>), grid, block, 0, s, a); break;
    }
    return hipGetLastError();
}

template <int L>
static hipError_t step_sched_layout(const StepArgs &a, zero_dtype gdt, hipStream_t s)
{
    const bool small = a.n_chunks <= (L == 1 ? ZERO_SMALL_LAUNCH_CHUNKS_12B : ZERO_SMALL_LAUNCH_CHUNKS);
    if (gdt == ZERO_BF16)
        return small ? step_sched_dispatch<L, ZERO_BF16, true>(a, s)
                     : step_sched_dispatch<L, ZERO_BF16, false>(a, s);
    return small ? step_sched_dispatch<L, ZERO_FP32, true>(a, s)
                 : step_sched_dispatch<L, ZERO_FP32, false>(a, s);
}

hipError_t launch_step_sched(const StepArgs &a, zero_dtype gdt, StateLayout layout, hipStream_t s)
{
    switch (layout) {
    case StateLayout::Fp32: return step_sched_layout<0>(a, gdt, s);
    case StateLayout::Bf16Moments: return step_sched_layout<1>(a, gdt, s);
    case StateLayout::Kahan: return step_sched_layout<2>(a, gdt, s);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_index_advance(int64_t *index, int64_t n, hipStream_t s)
{
    hipLaunchKernelGGL(step_index_advance_kernel, dim3(1), dim3(64), 0, s, index, n);
    return hipGetLastError();
}

// The extended step picks its fold at launch: groups of 1 or of all N ranks
// are the flat order (KC = -1); groups of 4 or 8 (GPUs per node) have
// compiled folds for N in {8, 16, 32, 64}; any other grouping runs the
// run-time fold (KC = 0).
template <zero_dtype G, int NC, int W>
static void launch_ex_n(const StepArgs &a, int K, dim3 grid, dim3 block, hipStream_t s)
{
    constexpr int K8 = (NC % 8 == 0 && NC > 8) ? 8 : 0;
    constexpr int K4 = (NC % 4 == 0 && NC > 4) ? 4 : 0;
    if (K == 1 || K == a.red.n_ranks)
        hipLaunchKernelGGL((shard_step_kernel<G, NC, true, -1, W>), grid, block, 0, s, a);
    else if (K8 == 8 && K == 8)
        hipLaunchKernelGGL((shard_step_kernel<G, NC, true, K8, W>), grid, block, 0, s, a);
    else if (K4 == 4 && K == 4)
        hipLaunchKernelGGL((shard_step_kernel<G, NC, true, K4, W>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((shard_step_kernel<G, NC, true, 0, W>), grid, block, 0, s, a);
}

template <zero_dtype G, int W>
static hipError_t step_ex_dispatch(const StepArgs &a, hipStream_t s)
{
    dim3 grid(chunk_grid(a.n_chunks)), block(kStepBlock);
    const int K = a.red.group;
    switch (a.red.n_ranks) {
    case 1: launch_ex_n<G, 1, W>(a, K, grid, block, s); break;
    case 2: launch_ex_n<G, 2, W>(a, K, grid, block, s); break;
    case 4: launch_ex_n<G, 4, W>(a, K, grid, block, s); break;
    case 8: launch_ex_n<G, 8, W>(a, K, grid, block, s); break;
    case 16: launch_ex_n<G, 16, W>(a, K, grid, block, s); break;
    case 32: launch_ex_n<G, 32, W>(a, K, grid, block, s); break;
    case 64: launch_ex_n<G, 64, W>(a, K, grid, block, s); break;
    default:
        if (K == 1 || K == a.red.n_ranks)
            hipLaunchKernelGGL((shard_step_kernel<G, 0, true, -1, W>), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL((shard_step_kernel<G, 0, true, 0, W>), grid, block, 0, s, a);
        break;
    }
    return hipGetLastError();
}

template <zero_dtype G, bool SMALL>
static hipError_t step_m16_dispatch(const StepArgs &a, hipStream_t s)
{
    dim3 grid(chunk_grid(a.n_chunks)), block(kStepBlock);
    switch (a.red.n_ranks) {
    case 1: hipLaunchKernelGGL((shard_step_m16_kernel<G, 1, SMALL>), grid, block, 0, s, a); break;
    case 2: hipLaunchKernelGGL((shard_step_m16_kernel<G, 2, SMALL>), grid, block, 0, s, a); break;
    case 4: hipLaunchKernelGGL((shard_step_m16_kernel<G, 4, SMALL>), grid, block, 0, s, a); break;
    case 8: hipLaunchKernelGGL((shard_step_m16_kernel<G, 8, SMALL>), grid, block, 0, s, a); break;
    case 16: hipLaunchKernelGGL((shard_step_m16_kernel<G, 16, SMALL>), grid, block, 0, s, a); break;
    case 32: hipLaunchKernelGGL((shard_step_m16_kernel<G, 32, SMALL>), grid, block, 0, s, a); break;
    case 64: hipLaunchKernelGGL((shard_step_m16_kernel<G, 64, SMALL>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((shard_step_m16_kernel<G, 0, SMALL>), grid, block, 0, s, a); break;
    }
    return hipGetLastError();
}

template <zero_dtype G>
static hipError_t step_kahan_dispatch(const StepArgs &a, hipStream_t s)
{
    const dim3 grid(chunk_grid(a.n_chunks)), block(kStepBlock);
    switch (a.red.n_ranks) {
    case 1: hipLaunchKernelGGL((shard_step_kahan_kernel<G, 1>), grid, block, 0, s, a); break;
    case 2: hipLaunchKernelGGL((shard_step_kahan_kernel<G, 2>), grid, block, 0, s, a); break;
    case 4: hipLaunchKernelGGL((shard_step_kahan_kernel<G, 4>), grid, block, 0, s, a); break;
    case 8: hipLaunchKernelGGL((shard_step_kahan_kernel<G, 8>), grid, block, 0, s, a); break;
    case 16: hipLaunchKernelGGL((shard_step_kahan_kernel<G, 16>), grid, block, 0, s, a); break;
    case 32: hipLaunchKernelGGL((shard_step_kahan_kernel<G, 32>), grid, block, 0, s, a); break;
    case 64: hipLaunchKernelGGL((shard_step_kahan_kernel<G, 64>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((shard_step_kahan_kernel<G, 0>), grid, block, 0, s, a); break;
    }
    return hipGetLastError();
}

hipError_t launch_step_kahan(const StepArgs &a, zero_dtype gdt, hipStream_t s)
{
    return gdt == ZERO_BF16 ? step_kahan_dispatch<ZERO_BF16>(a, s) : step_kahan_dispatch<ZERO_FP32>(a, s);
}

hipError_t launch_step_m16(const StepArgs &a, zero_dtype gdt, hipStream_t s)
{
    const bool small = a.n_chunks <= ZERO_SMALL_LAUNCH_CHUNKS_12B;
    if (gdt == ZERO_BF16)
        return small ? step_m16_dispatch<ZERO_BF16, true>(a, s) : step_m16_dispatch<ZERO_BF16, false>(a, s);
    return small ? step_m16_dispatch<ZERO_FP32, true>(a, s) : step_m16_dispatch<ZERO_FP32, false>(a, s);
}

hipError_t launch_step_ex(const StepArgs &a, zero_dtype gdt, hipStream_t s)
{
    // the same occupancy rule as the 16-byte step (same structure); measured
    // with one accumulated micro-batch, N = 8 bf16, working set kept out of
    // the last-level cache as for the 16-byte step, one wave against two:
    // 2M-element shards 0.44 / 0.45, 4M 0.47 / 0.48, 8M 0.54-0.55 / 0.53-0.54,
    // 16M 0.60-0.64 / 0.63, 32M 0.65-0.68 / 0.66-0.67 of the bytes of the
    // step with its accumulator read; 256M 0.65-0.66 / 0.61
    const bool small = a.n_chunks <= ZERO_SMALL_LAUNCH_CHUNKS;
    if (gdt == ZERO_BF16)
        return small ? step_ex_dispatch<ZERO_BF16, 2>(a, s) : step_ex_dispatch<ZERO_BF16, 1>(a, s);
    return small ? step_ex_dispatch<ZERO_FP32, 2>(a, s) : step_ex_dispatch<ZERO_FP32, 1>(a, s);
}

template <zero_dtype G, int NC>
static void launch_acc_n(const AccArgs &a, int K, dim3 grid, dim3 block, hipStream_t s)
{
    if (K == 1 || K == a.red.n_ranks)
        hipLaunchKernelGGL((accumulate_kernel<G, NC, -1>), grid, block, 0, s, a);
    else if (NC % 8 == 0 && NC > 8 && K == 8)
        hipLaunchKernelGGL((accumulate_kernel<G, NC, (NC % 8 == 0 && NC > 8) ? 8 : 0>), grid, block, 0, s, a);
    else if (NC % 4 == 0 && NC > 4 && K == 4)
        hipLaunchKernelGGL((accumulate_kernel<G, NC, (NC % 4 == 0 && NC > 4) ? 4 : 0>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((accumulate_kernel<G, NC, 0>), grid, block, 0, s, a);
}

template <zero_dtype G>
static hipError_t accumulate_dispatch(const AccArgs &a, hipStream_t s)
{
    dim3 grid(chunk_grid((a.n + kAccSpan - 1) / kAccSpan)), block(kStepBlock);
    const int K = a.red.group;
    switch (a.red.n_ranks) {
    case 1: launch_acc_n<G, 1>(a, K, grid, block, s); break;
    case 2: launch_acc_n<G, 2>(a, K, grid, block, s); break;
    case 4: launch_acc_n<G, 4>(a, K, grid, block, s); break;
    case 8: launch_acc_n<G, 8>(a, K, grid, block, s); break;
    case 16: launch_acc_n<G, 16>(a, K, grid, block, s); break;
    case 32: launch_acc_n<G, 32>(a, K, grid, block, s); break;
    case 64: launch_acc_n<G, 64>(a, K, grid, block, s); break;
    default:
        if (K == 1 || K == a.red.n_ranks)
            hipLaunchKernelGGL((accumulate_kernel<G, 0, -1>), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL((accumulate_kernel<G, 0, 0>), grid, block, 0, s, a);
        break;
    }
    return hipGetLastError();
}

hipError_t launch_accumulate(const AccArgs &a, zero_dtype gdt, hipStream_t s)
{
    return gdt == ZERO_BF16 ? accumulate_dispatch<ZERO_BF16>(a, s)
                            : accumulate_dispatch<ZERO_FP32>(a, s);
}

template <zero_dtype G>
static hipError_t reduce_dispatch(const ReduceArgs &a, hipStream_t s)
{
    dim3 grid(grid_for(a.n / Grad<G>::VEC + 1)), block(kBlock);
    switch (a.red.n_ranks) {
    case 1: hipLaunchKernelGGL((reduce_kernel<G, 1>), grid, block, 0, s, a); break;
    case 2: hipLaunchKernelGGL((reduce_kernel<G, 2>), grid, block, 0, s, a); break;
    case 4: hipLaunchKernelGGL((reduce_kernel<G, 4>), grid, block, 0, s, a); break;
    case 8: hipLaunchKernelGGL((reduce_kernel<G, 8>), grid, block, 0, s, a); break;
    case 16: hipLaunchKernelGGL((reduce_kernel<G, 16>), grid, block, 0, s, a); break;
    case 32: hipLaunchKernelGGL((reduce_kernel<G, 32>), grid, block, 0, s, a); break;
    case 64: hipLaunchKernelGGL((reduce_kernel<G, 64>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((reduce_kernel<G, 0>), grid, block, 0, s, a); break;
    }
    return hipGetLastError();
}

hipError_t launch_reduce(const ReduceArgs &a, zero_dtype gdt, hipStream_t s)
{
    return gdt == ZERO_BF16 ? reduce_dispatch<ZERO_BF16>(a, s) : reduce_dispatch<ZERO_FP32>(a, s);
}

hipError_t launch_adamw(const AdamArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL(adamw_kernel, dim3(grid_for(a.n / 4 + 1)), dim3(kBlock), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_gather(const GatherArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL(gather_kernel, dim3(chunk_grid(a.n_chunks)), dim3(kStepBlock), 0, s, a);
    return hipGetLastError();
}

}  // namespace zs
