// Clipping by the global gradient norm: the reduce with its sum of squares,
// sums of squares of many tensors, the coefficient, many tensors times the
// coefficient, and the clipped steps.
//
// All of it is streams: two operations an element for a sum of squares, one
// for a scaling, so the bound is HBM bandwidth and every load and store is 16
// bytes a lane.  A square is exact in double (an fp32 value has 24 bits), and
// the sums are kept in double: they can neither overflow nor lose small terms
// before some 2^29 equal ones, and the double pipe has room beside the stream.
//
// Sums without atomics: each workgroup (one wave) leaves one double, and one
// workgroup of a second launch adds those in a fixed order.  The order depends
// on the element count or the table alone, so results repeat bit for bit.

#include "zero_device.h"

namespace zs {

namespace {

constexpr int kFinishBlock = 1024;
constexpr int kFinishWaves = kFinishBlock / kStepLanes;

// The sum over the 64 lanes, in every lane: pairs, then pairs of pairs.
__device__ __forceinline__ double wave_sum(double x)
{
#pragma unroll
    for (int d = 1; d < kStepLanes; d *= 2)
        x = x + __shfl_xor(x, d);
    return x;
}

__device__ __forceinline__ double square_add(double x, double s) { return __builtin_fma(x, x, s); }

// norm and coefficient (zero_clip_coef in the header).  A sum that is not
// finite (it has an infinity or a NaN in it: finite fp32 squares cannot
// overflow a double's sum) makes the coefficient NaN.
__device__ __forceinline__ void write_clip(double sq, const ClipArgs &c)
{
    const double norm = c.inv_scale * __builtin_sqrt(sq);
    const double d = norm + c.eps;
    double coef = d <= c.max_norm ? c.inv_scale : c.inv_scale * (c.max_norm / d);
    if (!(sq < __builtin_inf()))
        coef = __builtin_nan("");
    c.out[0] = norm;
    c.out[1] = coef;
}

// ------------------------------------------------------- finishing the sums

// The sum of part[0 .. n) by a whole workgroup of kFinishBlock lanes: lane i
// adds part[i], part[i + kFinishBlock], ..., then the waves' sums are added in
// order.
__device__ __forceinline__ double block_sum(const double *part, int64_t n)
{
    __shared__ double waves[kFinishWaves];
    double s = 0.0;
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < n; i += kFinishBlock)
        s = s + part[i];
    s = wave_sum(s);
    if (threadIdx.x % kStepLanes == 0)
        waves[threadIdx.x / kStepLanes] = s;
    __syncthreads();
    double t = waves[0];
#pragma unroll
    for (int w = 1; w < kFinishWaves; ++w)
        t = t + waves[w];
    return t;
}

// Many partial sums become kFoldRuns first: workgroup b adds the b-th run of
// `run` of them.
constexpr int kFoldRuns = 256;

__global__ __launch_bounds__(kFinishBlock) void norm_fold_kernel(const double *part, int64_t n, int64_t run,
                                                                 double *out)
{
    const int64_t lo = blockIdx.x * run;
    const double s = block_sum(part + lo, n - lo < run ? n - lo : run);
    if (threadIdx.x == 0)
        out[blockIdx.x] = s;
}

// Tensor sums: the wave that meets a tensor's first piece adds its pieces.
__device__ __forceinline__ void tensor_sums(const FinishArgs &a, int64_t wave, int64_t n_waves)
{
    const int lane = threadIdx.x % kStepLanes;
    for (int64_t p = wave; p < a.n_part; p += n_waves) {
        int64_t count = a.pieces[p].tensor_pieces;
        const int64_t id = a.pieces[p].tensor_id;
        if (count <= 0 || id < 0 || id >= a.n_tensors)
            continue;
        if (count > a.n_part - p)
            count = a.n_part - p;
        double s = 0.0;
        for (int64_t i = lane; i < count; i += kStepLanes)
            s = s + a.part[p + i];
        s = wave_sum(s);
        if (lane == 0)
            a.tensor_sq[id] = s;
    }
}

// Workgroup 0 makes the total and the coefficient; the others, launched where
// they are asked for, the tensors' sums.
__global__ __launch_bounds__(kFinishBlock) void norm_finish_kernel(FinishArgs a)
{
    if (blockIdx.x > 0) {
        tensor_sums(a, (int64_t)(blockIdx.x - 1) * kFinishWaves + threadIdx.x / kStepLanes,
                    (int64_t)(gridDim.x - 1) * kFinishWaves);
        return;
    }
    const double s = block_sum(a.part, a.n_part);
    if (threadIdx.x == 0) {
        a.sq[0] = s;
        if (a.clip.out)
            write_clip(s, a.clip);
    }
}

__global__ __launch_bounds__(kStepLanes) void clip_coef_kernel(const double *sq, int64_t n, ClipArgs c)
{
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kStepLanes)
        s = s + sq[i];
    s = wave_sum(s);
    if (threadIdx.x == 0)
        write_clip(s, c);
}

// ------------------------------------------------------- reduce with the norm

// A wave pass takes a 16-byte load of each partial a lane: 512 elements of bf16
// (8 a lane), 256 of fp32 (4 a lane).  The reduced gradient leaves in rows of
// 256 elements, one 16-byte store a lane, so that each store instruction
// writes one run of 1 KiB; with bf16 partials a lane's 8 results first change
// places through LDS (two 16-byte stores a lane, each instruction writing
// every other 16 bytes, cost X).
constexpr int kRow = 4 * kStepLanes;

// Results e[0 .. VEC) of the group at 'lane' -> row r holds elements r * 256 +
// 4 * lane ... of the wave's pass.
template <int VEC>
__device__ __forceinline__ void to_rows(f32x4 *row, const float *e, f32x4 *lds, int lane)
{
    if constexpr (VEC == 4) {
        row[0] = (f32x4){e[0], e[1], e[2], e[3]};
    } else {
        lds[2 * lane] = (f32x4){e[0], e[1], e[2], e[3]};
        lds[2 * lane + 1] = (f32x4){e[4], e[5], e[6], e[7]};
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        row[0] = lds[lane];
        row[1] = lds[kStepLanes + lane];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// The two-level fold, one partial at a time: t sums a group of K in rank
// order, s the groups in order.  KC < 0: the flat order; KC > 0: K = KC, every
// test folding away where the ranks are unrolled; 0: K at run time.
template <int VEC, int KC> struct Fold {
    double s[VEC], t[VEC];
    int K, at = 0;
    bool some = false, begun = false;

    __device__ __forceinline__ explicit Fold(int k) : K(KC > 0 ? KC : k) {}
    __device__ __forceinline__ void close()
    {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            s[j] = some ? s[j] + t[j] : t[j];
        some = true;
    }
    template <zero_dtype G> __device__ __forceinline__ void add(u32x4 raw)
    {
        if constexpr (KC >= 0) {
            if (at == K) {
                close();
                at = 0;
            }
            if (at == 0)
                Grad<G>::first(t, raw);
            else
                Grad<G>::add(t, raw);
            ++at;
        } else {
            if (!begun)
                Grad<G>::first(t, raw);
            else
                Grad<G>::add(t, raw);
            begun = true;
        }
    }
    template <zero_dtype G, int B>
    __device__ __forceinline__ void batch(const PartialPtrs &pp, int k, int64_t i)
    {
        u32x4 raw[B];
#pragma unroll
        for (int j = 0; j < B; ++j)
            raw[j] = ld_raw(pp.p[k + j], i * Grad<G>::BYTES);
        __builtin_amdgcn_sched_barrier(0);   // every load of the batch in flight
#pragma unroll
        for (int j = 0; j < B; ++j)
            add<G>(raw[j]);
    }
};

// The sum over the ranks of a lane's word at element i, in s.  NC = 0: the
// number of ranks at run time, in batches of 8, 4, 2 and 1.
template <zero_dtype G, int NC, int KC, int VEC>
__device__ __forceinline__ void word_sum(double *s, const PartialPtrs &pp, int n, int K, int64_t i)
{
    Fold<VEC, KC> f(K);
    if constexpr (NC > 0) {
        constexpr int B = NC < kStepBatch ? NC : kStepBatch;
#pragma unroll
        for (int k = 0; k < NC; k += B)
            f.template batch<G, B>(pp, k, i);
    } else {
        int k = 0;
        for (; k + 8 <= n; k += 8)
            f.template batch<G, 8>(pp, k, i);
        if (n & 4) {
            f.template batch<G, 4>(pp, k, i);
            k += 4;
        }
        if (n & 2) {
            f.template batch<G, 2>(pp, k, i);
            k += 2;
        }
        if (n & 1)
            f.template batch<G, 1>(pp, k, i);
    }
    f.close();
#pragma unroll
    for (int j = 0; j < VEC; ++j)
        s[j] = f.s[j];
}

// One element by a whole wave, lane k loading partial k (there are at most 64):
// the loads take one round trip, the sum stays in rank order.
template <zero_dtype G>
__device__ __forceinline__ double wave_elem_sum(const PartialPtrs &pp, int n, int K, int64_t i)
{
    static_assert(ZERO_MAX_RANKS <= kStepLanes, "a lane a rank");
    const double mine = (int)threadIdx.x < n ? Grad<G>::one(pp.p[threadIdx.x], i) : 0.0;
    double s = 0.0, t = 0.0;
    for (int k = 0; k < n; ++k) {
        const double x = __shfl(mine, k);
        if (k % K == 0) {
            s = k == 0 ? s : (k == K ? t : s + t);
            t = x;
        } else {
            t = t + x;
        }
    }
    return n == K ? t : s + t;
}

// DIV: 1 multiplies by the exact reciprocal of a power of two, 2 divides.
template <zero_dtype G, int NC, int KC, int DIV>
__device__ __forceinline__ double reduce_norm_passes(const ReduceNormArgs &a, f32x4 *lds)
{
    constexpr int VEC = Grad<G>::VEC, ROWS = VEC / 4, PASS = VEC * kStepLanes;
    const int n = NC > 0 ? NC : a.red.n_ranks;
    const int lane = (int)threadIdx.x;
    const int64_t whole = a.n - a.n % VEC;   // the last n % VEC elements come after
    const int64_t first = (int64_t)blockIdx.x * a.passes * PASS;
    double sq = 0.0;
    for (int64_t at = first; at < first + a.passes * PASS && at < whole; at += PASS) {
        // past the end of the shard a lane reads its last group, and drops it
        const bool mine = at + VEC * lane < whole;
        const int64_t i = mine ? at + VEC * lane : whole - VEC;
        F32x<VEC> acc;
        if (a.acc)
            acc.load(a.acc + i);
        double s[VEC];
        word_sum<G, NC, KC, VEC>(s, a.parts, n, a.red.group, i);
        float g[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            if (a.acc)
                s[j] = (double)acc[j] + s[j];
            g[j] = DIV == 1 ? (float)(s[j] * a.red.inv_n) : (float)(s[j] / a.red.n);
            sq = square_add(mine ? (double)g[j] : 0.0, sq);
        }
        if (a.out) {
            f32x4 row[ROWS];
            to_rows<VEC>(row, g, lds, lane);
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const int64_t o = at + r * kRow + 4 * lane;
                if (o < whole)
                    st_nt((f32x4 *)(a.out + o), row[r]);
            }
        }
    }
    if (blockIdx.x == gridDim.x - 1) {
        for (int64_t e = whole; e < a.n; ++e) {
            double x = wave_elem_sum<G>(a.parts, n, a.red.group, e);
            if (a.acc)
                x = (double)a.acc[e] + x;
            const float g = finish_reduce<0>(x, a.red);
            if (lane == 0) {
                sq = square_add((double)g, sq);
                if (a.out)
                    a.out[e] = g;
            }
        }
    }
    return sq;
}

// W: resident waves per SIMD.
template <zero_dtype G, int NC, int KC, int W>
__global__ __launch_bounds__(kStepBlock) __attribute__((amdgpu_waves_per_eu(1, W)))
void reduce_norm_kernel(ReduceNormArgs a)
{
    __shared__ f32x4 lds[2 * kStepLanes];
    const double sq = wave_sum(a.red.pow2 ? reduce_norm_passes<G, NC, KC, 1>(a, lds)
                                          : reduce_norm_passes<G, NC, KC, 2>(a, lds));
    if (threadIdx.x == 0)
        a.part[blockIdx.x] = sq;
}

// ------------------------------------------------------- many tensors

// A piece starts at any multiple of its element size: 16-byte loads and
// stores at such an address, which gfx950 does in one access.
typedef u32x4 u32x4_any __attribute__((aligned(2)));

__device__ __forceinline__ u32x4 ld_any(const void *p)
{
    return __builtin_nontemporal_load((const u32x4_any *)p);
}

__device__ __forceinline__ double half_to_double(uint32_t h)
{
    return (double)(float)__builtin_bit_cast(_Float16, (uint16_t)h);
}

// VEC elements of one 16-byte word, widened.
template <int DT> struct Elem;

template <> struct Elem<ZERO_FP32> {
    static constexpr int VEC = 4, BYTES = 4;
    __device__ static __forceinline__ void widen(double *x, u32x4 r) { Grad<ZERO_FP32>::first(x, r); }
    __device__ static __forceinline__ double one(const void *p, int64_t i) { return (double)((const float *)p)[i]; }
    __device__ static __forceinline__ void put(void *p, int64_t i, double y) { ((float *)p)[i] = (float)y; }
};

template <> struct Elem<ZERO_BF16> {
    static constexpr int VEC = 8, BYTES = 2;
    __device__ static __forceinline__ void widen(double *x, u32x4 r) { Grad<ZERO_BF16>::first(x, r); }
    __device__ static __forceinline__ double one(const void *p, int64_t i)
    {
        return bf16_to_double(((const uint16_t *)p)[i]);
    }
    __device__ static __forceinline__ uint32_t narrow(double y) { return bf16_from_double(y); }
    __device__ static __forceinline__ void put(void *p, int64_t i, double y) { ((uint16_t *)p)[i] = (uint16_t)narrow(y); }
};

template <> struct Elem<ZERO_FP16> {
    static constexpr int VEC = 8, BYTES = 2;
    __device__ static __forceinline__ void widen(double *x, u32x4 r)
    {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            x[2 * q] = half_to_double(r[q] & 0xFFFFu);
            x[2 * q + 1] = half_to_double(r[q] >> 16);
        }
    }
    __device__ static __forceinline__ double one(const void *p, int64_t i)
    {
        return half_to_double(((const uint16_t *)p)[i]);
    }
    // double -> fp16 in one rounding, by way of fp32 rounded to odd, as
    // bf16_from_double (fp32 keeps 13 more bits than fp16, subnormals included)
    __device__ static __forceinline__ uint32_t narrow(double y)
    {
        const float f = (float)y;
        const double fd = (double)f;
        uint32_t u = __float_as_uint(f);
        if (__builtin_fabs(fd) > __builtin_fabs(y))
            u -= 1;
        if (fd != y)
            u |= 1;
        return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)__uint_as_float(u));
    }
    __device__ static __forceinline__ void put(void *p, int64_t i, double y) { ((uint16_t *)p)[i] = (uint16_t)narrow(y); }
};

// The descriptor of piece pi, with scalar loads (as chunk_at); a malformed one
// comes back empty.
__device__ __forceinline__ zero_piece piece_at(const zero_piece *table, int64_t pi)
{
    const char *p = (const char *)(table + __builtin_amdgcn_readfirstlane((int)pi));
    zero_piece c;
    c.src = (const void *)(uintptr_t)*(const_i64 *)(p + offsetof(zero_piece, src));
    c.dst = (void *)(uintptr_t)*(const_i64 *)(p + offsetof(zero_piece, dst));
    c.len = *(const_i32 *)(p + offsetof(zero_piece, len));
    const uint32_t dts = (uint32_t)*(const_i32 *)(p + offsetof(zero_piece, src_dt));
    c.src_dt = (int16_t)(dts & 0xFFFFu);
    c.dst_dt = (int16_t)(dts >> 16);
    c.tensor_id = 0;
    c.tensor_pieces = 0;
    if (c.len < 0 || c.len > (1 << 24) || !c.src)
        c.len = 0;
    return c;
}

// This lane's part of a piece's sum of squares: kNormUnroll loads of 16 bytes
// in flight, lanes past the end adding zeros.
constexpr int kNormWaves = 8;
constexpr int kNormUnroll = 1;
constexpr int kNormBlock = kNormWaves * kStepLanes;

template <int DT>
__device__ __forceinline__ double piece_square(const zero_piece &c)
{
    using E = Elem<DT>;
    const char *src = (const char *)c.src;
    const int words = c.len / E::VEC;
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    const int i = words * E::VEC + (int)threadIdx.x;
    if (i < c.len)
        s[0] = square_add(E::one(c.src, i), s[0]);
    for (int w0 = 0; w0 < words; w0 += kNormUnroll * kNormBlock) {
        u32x4 r[kNormUnroll];
#pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) {
            const int w = w0 + u * kNormBlock + (int)threadIdx.x;
            r[u] = w < words ? ld_any(src + (int64_t)w * 16) : (u32x4){0u, 0u, 0u, 0u};
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) {
            double x[E::VEC];
            E::widen(x, r[u]);
#pragma unroll
            for (int j = 0; j < E::VEC; ++j)
                s[j % 4] = square_add(x[j], s[j % 4]);
        }
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// A workgroup a piece.
__global__ __launch_bounds__(kNormBlock) void norm_pieces_kernel(PiecesArgs a)
{
    __shared__ double waves[2][kNormWaves];
    int side = 0;   // two sets of sums in turn: one barrier a piece is enough
    for (int64_t p = blockIdx.x; p < a.n_pieces; p += gridDim.x, side ^= 1) {
        const zero_piece c = piece_at(a.pieces, p);
        double s = 0.0;
        if (c.src_dt == ZERO_BF16)
            s = piece_square<ZERO_BF16>(c);
        else if (c.src_dt == ZERO_FP32)
            s = piece_square<ZERO_FP32>(c);
        else if (c.src_dt == ZERO_FP16)
            s = piece_square<ZERO_FP16>(c);
        s = wave_sum(s);
        if (threadIdx.x % kStepLanes == 0)
            waves[side][threadIdx.x / kStepLanes] = s;
        __syncthreads();
        if (threadIdx.x == 0) {
            double t = waves[side][0];
#pragma unroll
            for (int w = 1; w < kNormWaves; ++w)
                t = t + waves[side][w];
            a.part[p] = t;
        }
    }
}

// VEC elements (4 or 8) at any address their size divides, widened; and
// narrowed into an address aligned for all of them.
typedef u32x2 u32x2_any __attribute__((aligned(2)));

template <int S, int VEC> struct Load {
    static constexpr int BYTES = VEC * Elem<S>::BYTES;
    u32x4 r;
    __device__ __forceinline__ void get(const char *p)
    {
        if constexpr (BYTES == 16) {
            r = ld_any(p);
        } else {
            const u32x2 h = __builtin_nontemporal_load((const u32x2_any *)p);
            r = (u32x4){h.x, h.y, 0u, 0u};
        }
    }
    __device__ __forceinline__ void widen(double *x) const
    {
        double y[Elem<S>::VEC];
        Elem<S>::widen(y, r);
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            x[j] = y[j];
    }
};

template <int D, int VEC>
__device__ __forceinline__ void put_group(char *p, const double *y)
{
    if constexpr (D == ZERO_FP32) {
        static_assert(VEC == 4, "16 bytes of fp32");
        st_nt((f32x4 *)p, (f32x4){(float)y[0], (float)y[1], (float)y[2], (float)y[3]});
    } else {
        uint32_t w[VEC / 2];
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j)
            w[j] = Elem<D>::narrow(y[2 * j]) | (Elem<D>::narrow(y[2 * j + 1]) << 16);
        if constexpr (VEC == 8)
            st_nt((u32x4 *)p, (u32x4){w[0], w[1], w[2], w[3]});
        else
            st_nt((u32x2 *)p, (u32x2){w[0], w[1]});
    }
}

// coef times part `part` of a piece, then the parts kParts further on: a
// workgroup of kScaleWaves waves a part of kPartLen elements, each lane with
// kScaleUnroll groups in flight.  A lane's group is 8 elements where both types
// have 16 bits and 4 where one has 32, so that a wave's loads and its stores
// each cover one run of memory.  The stores are aligned: the elements before
// dst's first 16-byte boundary are done one by one, as is the end; the loads
// go by them, at any address.
constexpr int kScaleWaves = 8;
constexpr int kScaleUnroll = 2;
constexpr int kScaleBlock = kScaleWaves * kStepLanes;
constexpr int kParts = 2;
constexpr int kPartLen = 8192;

template <int S, int D>
__device__ __forceinline__ void scale_piece(const zero_piece &c, int part, double coef)
{
    using ES = Elem<S>;
    using ED = Elem<D>;
    constexpr int VEC = S == ZERO_FP32 || D == ZERO_FP32 ? 4 : 8;
    constexpr int U = kScaleUnroll;
    const int lane = (int)threadIdx.x;
    int head = (int)((16u - ((uintptr_t)c.dst & 15u)) & 15u) / ED::BYTES;
    if (head > c.len)
        head = c.len;
    const int groups = (c.len - head) / VEC;
    const char *src = (const char *)c.src + head * ES::BYTES;
    char *dst = (char *)c.dst + head * ED::BYTES;
    if (part == 0) {
        const int tail = head + groups * VEC;
        if (lane < head)
            ED::put(c.dst, lane, coef * ES::one(c.src, lane));
        if (tail + lane < c.len)
            ED::put(c.dst, tail + lane, coef * ES::one(c.src, tail + lane));
    }
    constexpr int PART = kPartLen / VEC, PASS = U * kScaleBlock;
    static_assert(PART % PASS == 0, "a part is whole passes");
    for (int p0 = part * PART; p0 < groups; p0 += kParts * PART) {
        for (int g0 = p0; g0 < p0 + PART && g0 < groups; g0 += PASS) {
            Load<S, VEC> r[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int g = g0 + u * kScaleBlock + lane;
                if (g < groups)
                    r[u].get(src + (int64_t)g * Load<S, VEC>::BYTES);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int g = g0 + u * kScaleBlock + lane;
                if (g < groups) {
                    double x[VEC];
                    r[u].widen(x);
#pragma unroll
                    for (int j = 0; j < VEC; ++j)
                        x[j] = coef * x[j];
                    put_group<D, VEC>(dst + (int64_t)g * (VEC * ED::BYTES), x);
                }
            }
        }
    }
}

template <int S>
__device__ __forceinline__ void scale_to(const zero_piece &c, int part, double coef)
{
    if (c.dst_dt == ZERO_BF16)
        scale_piece<S, ZERO_BF16>(c, part, coef);
    else if (c.dst_dt == ZERO_FP32)
        scale_piece<S, ZERO_FP32>(c, part, coef);
    else if (c.dst_dt == ZERO_FP16)
        scale_piece<S, ZERO_FP16>(c, part, coef);
}

// The parts of a run of kPieceRun pieces come one after the other, so that the
// workgroups that short pieces leave without work lie side by side (every
// second workgroup idle had slowed the rest of some types to half).
constexpr int kPieceRun = 64;

__global__ __launch_bounds__(kScaleBlock) void scale_pieces_kernel(PiecesArgs a)
{
    const double coef = ((const const_f64 *)a.clip)[1];
    if (!(coef == coef))
        return;
    const int part = (int)(blockIdx.x / kPieceRun % kParts);
    const int64_t first = (int64_t)(blockIdx.x / (kPieceRun * kParts)) * kPieceRun + blockIdx.x % kPieceRun;
    for (int64_t p = first; p < a.n_pieces; p += gridDim.x / kParts) {
        const zero_piece c = piece_at(a.pieces, p);
        if (c.len == 0 || !c.dst || (coef == 1.0 && c.dst == c.src && c.dst_dt == c.src_dt))
            continue;
        if (c.src_dt == ZERO_BF16)
            scale_to<ZERO_BF16>(c, part, coef);
        else if (c.src_dt == ZERO_FP32)
            scale_to<ZERO_FP32>(c, part, coef);
        else if (c.src_dt == ZERO_FP16)
            scale_to<ZERO_FP16>(c, part, coef);
    }
}

// ------------------------------------------------------- the clipped steps

// Resident waves per SIMD, as the steps that do not clip.
template <int L, zero_dtype G, int NC, bool SMALL>
constexpr int kClipWaves = L == 0 ? (SMALL ? 2 : 1)
                                  : (L == 1 ? kM16Waves<G, NC, SMALL> : kKahanWaves);

// L, SMALL: as the scheduled steps.  The coefficient and, for a scheduled
// step, the constants are read when the kernel runs.
template <int L, zero_dtype G, int NC, bool SMALL>
__global__ __launch_bounds__(kStepBlock) __attribute__((amdgpu_waves_per_eu(1, kClipWaves<L, G, NC, SMALL>)))
void shard_step_clip_kernel(StepArgs a)
{
    const double coef = ((const const_f64 *)a.clip)[1];
    if (!(coef == coef))
        return;
    StepScalars k = a.k;
    if (a.sched) {
        const int64_t t = *(const_i64 *)a.sched_index;
        if (t < 0 || t >= a.n_sched)
            return;
        const const_f64 *e = (const const_f64 *)(a.sched + t);
        k.b1 = e[0]; k.c1 = e[1]; k.b2 = e[2]; k.c2 = e[3]; k.bc1 = e[4]; k.bc2 = e[5];
        k.eps = e[6]; k.lr = e[7]; k.dec = e[8]; k.wd = e[9];
    }
    for (int64_t ci = blockIdx.x; ci < a.n_chunks; ci += gridDim.x) {
        if constexpr (L == 0)
            step_chunk<G, NC, false, -1, 0, true>(a, chunk_at(a.chunks, ci), k, coef);
        else if constexpr (L == 1)
            step_chunk_m16<G, NC, SMALL, true>(a, chunk_at(a.chunks, ci), k, coef);
        else
            step_chunk_kahan<G, NC, true>(a, chunk_at(a.chunks, ci), k, coef);
    }
}

// ------------------------------------------------------- launchers

// Workgroups of `block` lanes for `want` units of work, which stride: a power of
// two at most, and fewer than 2^32 work-items.
unsigned block_grid(int64_t want, int block)
{
    const int64_t most = (int64_t(1) << 31) / block;
    return (unsigned)(want < most ? want : most);
}

// More partial sums than this are folded before they are finished.
constexpr int64_t kFoldFrom = 16384;

hipError_t finish(const FinishArgs &f, hipStream_t s)
{
    unsigned grid = 1;
    if (f.tensor_sq && f.n_part > 0) {
        const int64_t want = (f.n_part + kFinishWaves - 1) / kFinishWaves;
        grid += (unsigned)(want < 1024 ? want : 1024);
    }
    hipLaunchKernelGGL(norm_finish_kernel, dim3(grid), dim3(kFinishBlock), 0, s, f);
    return hipGetLastError();
}

template <zero_dtype G, int NC, int W>
void launch_reduce_norm_n(const ReduceNormArgs &a, int K, dim3 grid, hipStream_t s)
{
    const dim3 block(kStepBlock);
    constexpr int K8 = (NC % 8 == 0 && NC > 8) ? 8 : 0;
    constexpr int K4 = (NC % 4 == 0 && NC > 4) ? 4 : 0;
    if (K == 1 || K == a.red.n_ranks)
        hipLaunchKernelGGL((reduce_norm_kernel<G, NC, -1, W>), grid, block, 0, s, a);
    else if (K8 == 8 && K == 8)
        hipLaunchKernelGGL((reduce_norm_kernel<G, NC, K8, W>), grid, block, 0, s, a);
    else if (K4 == 4 && K == 4)
        hipLaunchKernelGGL((reduce_norm_kernel<G, NC, K4, W>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((reduce_norm_kernel<G, NC, 0, W>), grid, block, 0, s, a);
}

template <zero_dtype G>
hipError_t reduce_norm_dispatch(const ReduceNormArgs &a, dim3 grid, hipStream_t s)
{
    const int K = a.red.group;
    switch (a.red.n_ranks) {
    case 1: launch_reduce_norm_n<G, 1, 8>(a, K, grid, s); break;
    case 2: launch_reduce_norm_n<G, 2, 8>(a, K, grid, s); break;
    case 4: launch_reduce_norm_n<G, 4, 4>(a, K, grid, s); break;
    case 8: launch_reduce_norm_n<G, 8, 2>(a, K, grid, s); break;
    case 16: launch_reduce_norm_n<G, 16, 2>(a, K, grid, s); break;
    case 32: launch_reduce_norm_n<G, 32, 1>(a, K, grid, s); break;
    case 64: launch_reduce_norm_n<G, 64, 1>(a, K, grid, s); break;
    default:
        if (a.red.n_ranks < 8)
            launch_reduce_norm_n<G, 0, 4>(a, K, grid, s);
        else
            launch_reduce_norm_n<G, 0, 2>(a, K, grid, s);
        break;
    }
    return hipGetLastError();
}

template <int L, zero_dtype G, bool SMALL>
hipError_t step_clip_dispatch(const StepArgs &a, hipStream_t s)
{
    const dim3 grid(chunk_grid(a.n_chunks)), block(kStepBlock);
    switch (a.red.n_ranks) {
    case 1: hipLaunchKernelGGL((shard_step_clip_kernel<L, G, 1, SMALL>), grid, block, 0, s, a); break;
    case 2: hipLaunchKernelGGL((shard_step_clip_kernel<L, G, 2, SMALL>), grid, block, 0, s, a); break;
    case 4: hipLaunchKernelGGL((shard_step_clip_kernel<L, G, 4, SMALL>), grid, block, 0, s, a); break;
    case 8: hipLaunchKernelGGL((shard_step_clip_kernel<L, G, 8, SMALL>), grid, block, 0, s, a); break;
    case 16: hipLaunchKernelGGL((shard_step_clip_kernel<L, G, 16, SMALL>), grid, block, 0, s, a); break;
    case 32: hipLaunchKernelGGL((shard_step_clip_kernel<L, G, 32, SMALL>), grid, block, 0, s, a); break;
    case 64: hipLaunchKernelGGL((shard_step_clip_kernel<L, G, 64, SMALL>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((shard_step_clip_kernel<L, G, 0, SMALL>), grid, block, 0, s, a); break;
    }
    return hipGetLastError();
}

template <int L>
hipError_t step_clip_layout(const StepArgs &a, zero_dtype gdt, hipStream_t s)
{
    const bool small = a.n_chunks <= (L == 1 ? ZERO_SMALL_LAUNCH_CHUNKS_12B : ZERO_SMALL_LAUNCH_CHUNKS);
    if (gdt == ZERO_BF16)
        return small ? step_clip_dispatch<L, ZERO_BF16, true>(a, s)
                     : step_clip_dispatch<L, ZERO_BF16, false>(a, s);
    return small ? step_clip_dispatch<L, ZERO_FP32, true>(a, s)
                 : step_clip_dispatch<L, ZERO_FP32, false>(a, s);
}

}  // namespace

hipError_t launch_reduce_norm(ReduceNormArgs a, zero_dtype gdt, FinishArgs f, hipStream_t s)
{
    f.part = a.part;
    f.n_part = reduce_norm_waves(a.n, gdt, &a.passes);
    if (f.n_part > 0) {
        const dim3 grid((unsigned)f.n_part);
        const hipError_t e = gdt == ZERO_BF16 ? reduce_norm_dispatch<ZERO_BF16>(a, grid, s)
                                              : reduce_norm_dispatch<ZERO_FP32>(a, grid, s);
        if (e != hipSuccess)
            return e;
    }
    if (f.n_part > kFoldFrom) {
        const int64_t run = (f.n_part + kFoldRuns - 1) / kFoldRuns;
        double *out = a.part + f.n_part;
        const int64_t runs = (f.n_part + run - 1) / run;
        hipLaunchKernelGGL(norm_fold_kernel, dim3((unsigned)runs), dim3(kFinishBlock), 0, s, f.part,
                           f.n_part, run, out);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
        f.part = out;
        f.n_part = runs;
    }
    return finish(f, s);
}

int64_t reduce_norm_waves(int64_t n, zero_dtype gdt, int64_t *passes)
{
    const int64_t pass = kStepLanes * (gdt == ZERO_BF16 ? Grad<ZERO_BF16>::VEC : Grad<ZERO_FP32>::VEC);
    const int64_t all = (n + pass - 1) / pass;
    *passes = (all + ZERO_NORM_PARTIALS - 1) / ZERO_NORM_PARTIALS;
    return all ? (all + *passes - 1) / *passes : 0;
}

int64_t reduce_norm_workspace(int64_t n, zero_dtype gdt)
{
    int64_t passes;
    const int64_t waves = reduce_norm_waves(n, gdt, &passes);
    return 8 * (waves + (waves > kFoldFrom ? kFoldRuns : 0));
}

hipError_t launch_clip_coef(const double *sq, int64_t n, const ClipArgs &c, hipStream_t s)
{
    hipLaunchKernelGGL(clip_coef_kernel, dim3(1), dim3(kStepLanes), 0, s, sq, n, c);
    return hipGetLastError();
}

hipError_t launch_norm_pieces(const PiecesArgs &a, FinishArgs f, hipStream_t s)
{
    f.part = a.part;
    f.n_part = a.n_pieces;
    f.pieces = a.pieces;
    if (a.n_pieces > 0) {
        hipLaunchKernelGGL(norm_pieces_kernel, dim3(block_grid(a.n_pieces, kNormBlock)), dim3(kNormBlock), 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return finish(f, s);
}

hipError_t launch_scale_pieces(const PiecesArgs &a, hipStream_t s)
{
    const int64_t runs = (a.n_pieces + kPieceRun - 1) / kPieceRun;
    const dim3 grid(block_grid(runs * kPieceRun * kParts, kScaleBlock));
    hipLaunchKernelGGL(scale_pieces_kernel, grid, dim3(kScaleBlock), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_step_clipped(const StepArgs &a, zero_dtype gdt, StateLayout layout, hipStream_t s)
{
    switch (layout) {
    case StateLayout::Fp32: return step_clip_layout<0>(a, gdt, s);
    case StateLayout::Bf16Moments: return step_clip_layout<1>(a, gdt, s);
    case StateLayout::Kahan: return step_clip_layout<2>(a, gdt, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace zs
