// Low-rank adapters of many requests beside a shared projection:
//
//   y[b] = base[b] + f_e (x[b] A_e^T) B_e^T,   e the adapter of row b,
//
// A_e [r_e][K], B_e [N][r_e] in bf16, as checkpoints hold them.  Rows are taken
// in tiles of up to 64 rows of one adapter, in the order that adapter_rows made
// once for all projections of a step.
//
// Two launches.  Down: a workgroup owns a tile and a piece of K; its eight waves
// take 64 elements of K in turn, A's rows the one operand of the matrix cores, the
// x rows the other, both straight from memory (each is read once by a tile); the
// partial sums go to the workspace in fp32.  Up: a workgroup owns a tile and 256
// columns of y, adds the pieces in order and multiplies by B.  For many rows a
// launch between them adds the pieces up.  Everything between the operands is fp32:
// x as fp32 enters as three bf16 terms that hold it exactly, codes are exact in
// bf16, and the sums between the two products enter the second as two terms (17
// bits) for bf16 outputs and three (exact) for fp32.
//
// Few rows: the time is latency.  The workgroups' first loads depend on each other
// (the tile; the adapter's addresses and rank and the rows; the operands), three
// times a miss to memory in either launch, since the caches of the XCDs start empty.
// So nothing else may wait: operands come through unconditional loads (branches
// around them made each wait for itself: 64 rows of one adapter, rank 16, the second
// launch 15.8 -> 9.6 us).  Both products in one launch, each workgroup with the
// tile's sums over all of K for itself, was slower (16 rows: 10.4 against 8.1 us, 7.4 by
// now; 70 rows, K = 17408: 49 against 12): a CU reads some 27 KB a microsecond so.
#include <type_traits>

#include "layer.h"

namespace qg {

constexpr int AD_CHUNK = 64;  // ranks a workgroup takes at a time
constexpr int AD_WAVES = 8;   // of a workgroup of the first product
constexpr int AD_UP = 4;      // waves of a workgroup of the second, 64 columns each

struct Tile {
    int e, first, n;
};

// Record i of the order; false where there is none or it breaks its rules.
__device__ __forceinline__ bool tile_of(const AdaptArgs &a, int i, Tile *t, bool report)
{
    // both loads on their way at once: record i exists for every workgroup of the grid
    const int4 head = *(const int4 *)a.plan, r = ((const int4 *)a.plan)[1 + i];
    if (head.y != a.B || head.z != a.E) {
        if (report)
            __hip_atomic_fetch_or(a.status, DEV_BAD_ADAPTER, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        return false;
    }
    if (i >= head.x)
        return false;
    t->e = __builtin_amdgcn_readfirstlane(r.x);
    t->first = __builtin_amdgcn_readfirstlane(r.y);
    t->n = __builtin_amdgcn_readfirstlane(r.z);
    if (t->e < 0 || t->e > a.E || t->n < 1 || t->n > AD_ROWS || t->first < 0 || t->first > a.B - t->n) {
        if (report)
            __hip_atomic_fetch_or(a.status, DEV_BAD_ADAPTER, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        return false;
    }
    return true;
}

// The rank of adapter e; 0 for rows without one and where it breaks its rules.
__device__ __forceinline__ int rank_of(const AdaptArgs &a, int e, bool report)
{
    if (e >= a.E)
        return 0;
    const int r = a.ranks ? __builtin_amdgcn_readfirstlane(a.ranks[e]) : a.rank;
    if (r < 0 || r > a.rank || (r & 7)) {
        if (report)
            __hip_atomic_fetch_or(a.status, DEV_BAD_ADAPTER, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        return 0;
    }
    return r;
}

__device__ __forceinline__ const int *rows_of(const AdaptArgs &a)
{
    return a.plan + 4 + 4 * adapter_tiles(a.B, a.E);
}

// ------------------------------------------------------------------- down

template <int ACT>
struct XTerms {
    static constexpr int N = ACT == ACT_F32 ? 3 : 1;
};

// Eight elements of a row of x as they are in memory.
template <int ACT>
struct XRaw {
    static constexpr int REGS = ACT == ACT_F32 ? 8 : ACT == ACT_BF16 ? 4 : 2;
    uint32_t r[REGS];
    __device__ __forceinline__ void load(const uint8_t *row, int k)
    {
        __builtin_memcpy(r, row + (int64_t)k * REGS / 2, 4 * REGS);
    }
    __device__ __forceinline__ Split<XTerms<ACT>::N> operand() const
    {
        Split<XTerms<ACT>::N> s;
        if constexpr (ACT == ACT_F32) {
            float f[8];
            __builtin_memcpy(f, r, 32);
            s = split_f32<3>(f);
        } else if constexpr (ACT == ACT_BF16) {
            __builtin_memcpy(&s.t[0], r, 16);
        } else {
            s.t[0] = q8_to_bf16(r[0], r[1]);
        }
        return s;
    }
};

// The first n of eight elements made zeros.
__device__ __forceinline__ bf16x8 drop_first(bf16x8 v, int n)
{
    u32x4 r = __builtin_bit_cast(u32x4, v);
#pragma unroll
    for (int i = 0; i < 4; i++)
        r[i] = 2 * i + 1 < n ? 0u : 2 * i < n ? r[i] & 0xFFFF0000u : r[i];
    return __builtin_bit_cast(bf16x8, r);
}

// RT tiles of 16 ranks from r0, CT tiles of 16 rows; k0 .. k1-1 of K.
template <int ACT, int RT, int CT>
__device__ __forceinline__ void down_tile(const AdaptArgs &a, const Tile &t, int rank, int r0, int k0, int k1, int piece,
                                          f32x4 *red)
{
    constexpr int NT = XTerms<ACT>::N;
    constexpr int ESZ = ACT == ACT_F32 ? 4 : ACT == ACT_BF16 ? 2 : 1;
    const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m = lane & 15, kg = (lane >> 4) * 8;
    const int *rows = rows_of(a);
    const uint8_t *xp[CT];
#pragma unroll
    for (int c = 0; c < CT; c++) {
        const int i = t.first + min(c * 16 + m, t.n - 1);
        int row = rows[i];
        row = row < 0 || row >= a.B ? 0 : row;  // reported and not written by the second launch
        xp[c] = (const uint8_t *)a.x + (int64_t)row * a.ldx * ESZ;
    }
    const __bf16 *A = (const __bf16 *)uniform_ptr(a.a_table[t.e]);
    const __bf16 *ap[RT];
#pragma unroll
    for (int r = 0; r < RT; r++)
        ap[r] = A + (int64_t)min(r0 + r * 16 + m, rank - 1) * a.K;

    f32x4 acc[RT][CT];
#pragma unroll
    for (int r = 0; r < RT; r++)
#pragma unroll
        for (int c = 0; c < CT; c++)
            acc[r][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    // 64 elements a wave and turn: whole lines of bf16 rows
    int k = k0 + wid * 64;
    for (; k + 64 <= k1; k += AD_WAVES * 64) {
        bf16x8 w[2][RT];
        XRaw<ACT> xr[2][CT];
#pragma unroll
        for (int s = 0; s < 2; s++) {
            const int at = k + s * 32 + kg;
#pragma unroll
            for (int r = 0; r < RT; r++)
                __builtin_memcpy(&w[s][r], ap[r] + at, 16);
#pragma unroll
            for (int c = 0; c < CT; c++)
                xr[s][c].load(xp[c], at);
        }
        __builtin_amdgcn_sched_barrier(0);  // every load before the first product
#pragma unroll
        for (int s = 0; s < 2; s++)
#pragma unroll
            for (int c = 0; c < CT; c++) {
                const Split<NT> xs = xr[s][c].operand();
#pragma unroll
                for (int q = 0; q < NT; q++)
#pragma unroll
                    for (int r = 0; r < RT; r++)
                        acc[r][c] = mfma(w[s][r], xs.t[q], acc[r][c]);
            }
    }
    // the partial turn of the row's end: vectors that would pass it are the row's last
    // eight elements, those of the vector before made zeros on both sides (loads in
    // branches would each wait for themselves: K = 5119 took 10.2 us where 5120 took 7.9)
    k = k0 + ((k1 - k0) & ~63);
    if (k < k1 && ((k - k0) >> 6) % AD_WAVES == wid) {
        bf16x8 w[2][RT];
        XRaw<ACT> xr[2][CT];
        int skip[2];
#pragma unroll
        for (int s = 0; s < 2; s++) {
            const int want = k + s * 32 + kg, at = min(want, a.K - 8);
            skip[s] = want - at;
#pragma unroll
            for (int r = 0; r < RT; r++)
                __builtin_memcpy(&w[s][r], ap[r] + at, 16);
#pragma unroll
            for (int c = 0; c < CT; c++)
                xr[s][c].load(xp[c], at);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < 2; s++) {
#pragma unroll
            for (int r = 0; r < RT; r++)
                w[s][r] = drop_first(w[s][r], skip[s]);
#pragma unroll
            for (int c = 0; c < CT; c++) {
                const Split<NT> xs = xr[s][c].operand();
#pragma unroll
                for (int q = 0; q < NT; q++) {
                    const bf16x8 v = drop_first(xs.t[q], skip[s]);
#pragma unroll
                    for (int r = 0; r < RT; r++)
                        acc[r][c] = mfma(w[s][r], v, acc[r][c]);
                }
            }
        }
    }

    // the waves' sums meet in LDS, the upper four's added to the lower's first (64 KB
    // for eight waves), and go to the workspace
    auto put = [&](int w) {
#pragma unroll
        for (int r = 0; r < RT; r++)
#pragma unroll
            for (int c = 0; c < CT; c++)
                red[((r * CT + c) * 4 + w) * 64 + lane] = acc[r][c];
    };
    if (wid >= 4)
        put(wid - 4);
    __syncthreads();
    if (wid < 4) {
#pragma unroll
        for (int r = 0; r < RT; r++)
#pragma unroll
            for (int c = 0; c < CT; c++)
                acc[r][c] += red[((r * CT + c) * 4 + wid) * 64 + lane];
        put(wid);  // its own places
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RT * CT; i++) {
        if (i % AD_WAVES != wid)
            continue;
        const int r = i / CT, c = i % CT;
        f32x4 s = red[(i * 4 + 0) * 64 + lane];
#pragma unroll
        for (int w = 1; w < 4; w++)
            s += red[(i * 4 + w) * 64 + lane];
        const int col = c * 16 + m, at = r0 + r * 16 + (lane >> 4) * 4;
        if (col < t.n && at < rank) {  // rank is a multiple of 8
            if constexpr (ACT == ACT_CODES) {
                const int row = rows[t.first + col];
                const float sc = row < 0 || row >= a.B ? 0.f : a.xs[row];
#pragma unroll
                for (int j = 0; j < 4; j++)
                    s[j] *= sc;
            }
            *(f32x4 *)(a.part + ((int64_t)piece * a.B + t.first + col) * a.ldp + at) = s;
        }
    }
}

template <int ACT>
__global__ __launch_bounds__(64 * AD_WAVES) void adapt_down_kernel(AdaptArgs a, int chunks)
{
    __shared__ f32x4 red[4 * 4 * 4 * 64];  // 64 KB
    const int piece = blockIdx.x % a.split, rest = blockIdx.x / a.split;
    Tile t;
    if (!tile_of(a, rest / chunks, &t, false))
        return;
    const int rank = rank_of(a, t.e, false), r0 = rest % chunks * AD_CHUNK;
    if (r0 >= rank)
        return;
    const int k0 = piece * a.kc, k1 = min(k0 + a.kc, a.K);
    const int left = rank - r0;
    if (t.n <= 16) {
        if (left <= 16) down_tile<ACT, 1, 1>(a, t, rank, r0, k0, k1, piece, red);
        else if (left <= 32) down_tile<ACT, 2, 1>(a, t, rank, r0, k0, k1, piece, red);
        else down_tile<ACT, 4, 1>(a, t, rank, r0, k0, k1, piece, red);
    } else if (t.n <= 32) {
        if (left <= 16) down_tile<ACT, 1, 2>(a, t, rank, r0, k0, k1, piece, red);
        else if (left <= 32) down_tile<ACT, 2, 2>(a, t, rank, r0, k0, k1, piece, red);
        else down_tile<ACT, 4, 2>(a, t, rank, r0, k0, k1, piece, red);
    } else {
        if (left <= 16) down_tile<ACT, 1, 4>(a, t, rank, r0, k0, k1, piece, red);
        else if (left <= 32) down_tile<ACT, 2, 4>(a, t, rank, r0, k0, k1, piece, red);
        else down_tile<ACT, 4, 4>(a, t, rank, r0, k0, k1, piece, red);
    }
}

// --------------------------------------------------------------------- up

template <int OUTT>
struct UpTerms {
    static constexpr int N = OUTT == OUT_F32 ? 3 : 2;
};

// Sixteen neighbouring outputs of a lane.
template <int OUTT>
struct Out16 {
    static constexpr int NW = OUTT == OUT_F32 ? 4 : 2;
    u32x4 w[NW];
    __device__ __forceinline__ void load(const void *p) { __builtin_memcpy(w, p, 16 * NW); }
    // The outputs from the d-th on; those behind them are anything.
    __device__ __forceinline__ void move_down(int d)
    {
        constexpr int PER = OUTT == OUT_F32 ? 1 : 2, WORDS = 16 / PER;  // outputs a word, words
        uint32_t v[WORDS];
#pragma unroll
        for (int i = 0; i < WORDS; i++)
            v[i] = w[i / 4][i % 4];
        // by masks: of selections the compiler makes places that the lane computes
#pragma unroll
        for (int step = WORDS / 2; step; step >>= 1) {
            const uint32_t m = (d / PER) & step ? 0xFFFFFFFFu : 0u;
#pragma unroll
            for (int i = 0; i + step < WORDS; i++)
                v[i] = (v[i + step] & m) | (v[i] & ~m);
        }
        if constexpr (PER == 2) {
            const uint32_t sh = d & 1 ? 16 : 0;
#pragma unroll
            for (int i = 0; i < WORDS; i++)
                v[i] = __builtin_amdgcn_alignbit(v[i + 1 < WORDS ? i + 1 : i], v[i], sh);
        }
#pragma unroll
        for (int i = 0; i < WORDS; i++)
            w[i / 4][i % 4] = v[i];
    }
    __device__ __forceinline__ float at(int i) const
    {
        if constexpr (OUTT == OUT_F32)
            return __uint_as_float(w[i / 4][i % 4]);
        else
            return __uint_as_float(i & 1 ? w[i / 8][i % 8 / 2] & 0xFFFF0000u : w[i / 8][i % 8 / 2] << 16);
    }
};

// K outputs of v to p, and the rest of v moved to its front.
template <int OUTT, int K>
__device__ __forceinline__ void store_some(uint8_t **p, float *v)
{
    if constexpr (OUTT == OUT_F32) {
        __builtin_memcpy(*p, v, 4 * K);
        *p += 4 * K;
    } else {
        __bf16 h[K];
#pragma unroll
        for (int i = 0; i < K; i++)
            h[i] = (__bf16)v[i];
        __builtin_memcpy(*p, h, 2 * K);
        *p += 2 * K;
    }
#pragma unroll
    for (int i = 0; i + K < 16; i++)
        v[i] = v[i + K];
}

// Sixteen neighbouring outputs, or the `left` that are there: in pieces of powers of
// two, since fifteen stores of elements are so many instructions that fetching them
// takes longer than all else (70 rows of 5104 instead of 5120 fp32 outputs: 22 us
// instead of 12).
template <int OUTT>
__device__ __forceinline__ void store16(void *to, int left, float *v)
{
    uint8_t *p = (uint8_t *)to;
    if (left >= 16) {
        store_some<OUTT, 16>(&p, v);
        return;
    }
    if (left & 8)
        store_some<OUTT, 8>(&p, v);
    if (left & 4)
        store_some<OUTT, 4>(&p, v);
    if (left & 2)
        store_some<OUTT, 2>(&p, v);
    if (left & 1)
        store_some<OUTT, 1>(&p, v);
}

// Eight ranks of a row of the sums between the products: the pieces in order.
__device__ __forceinline__ void low_sum(const AdaptArgs &a, int row, int at, int rank, float *v)
{
#pragma unroll
    for (int j = 0; j < 8; j++)
        v[j] = 0.f;
    if (at < rank) {
        const float *p = a.part + (int64_t)row * a.ldp + at;
        const int64_t step = (int64_t)a.B * a.ldp;
#pragma unroll 8
        for (int s = 0; s < a.split; s++) {
            const f32x4 lo = *(const f32x4 *)(p + s * step), hi = *(const f32x4 *)(p + s * step + 4);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                v[j] += lo[j];
                v[4 + j] += hi[j];
            }
        }
    }
}

// join: the sums as the bf16 terms that the second product takes, [term][row][ldk],
// in the sorted order of the rows; zeros from an adapter's rank to ldk.  Eight
// ranks a thread, 16 rows a workgroup.
template <int NT>
__global__ __launch_bounds__(128) void adapt_join_kernel(AdaptArgs a)
{
    Tile t;
    if (!tile_of(a, blockIdx.x >> 2, &t, false))
        return;
    const int rank = rank_of(a, t.e, false);
    if (rank == 0)
        return;
    const float f = a.factors ? a.factors[t.e] : 1.f;
    const int groups = a.ldk >> 3;
    const int r0 = (blockIdx.x & 3) * 16, n = min(t.n - r0, 16);
    for (int i = threadIdx.x; i < n * groups; i += 128) {
        const int row = t.first + r0 + i / groups, at = i % groups * 8;
        float v[8];
        low_sum(a, row, at, rank, v);
#pragma unroll
        for (int j = 0; j < 8; j++)
            v[j] *= f;
        const Split<NT> s = split_f32<NT>(v);
#pragma unroll
        for (int q = 0; q < NT; q++)
            *(bf16x8 *)(a.low + ((int64_t)q * a.B + row) * a.ldk + at) = s.t[q];
    }
}

// Whether all columns of a workgroup are there, or it holds a row's end, loaded from
// the row's last sixteen outputs.
enum { COLS_ALL, COLS_END };

// up: CT tiles of 16 rows times 64 columns a wave.  The B rows of the four matrix
// tiles are taken so that a lane's sixteen sums are neighbours in y.  JOINED: the
// sums between the products come as terms from the join, else each workgroup adds
// its tile's pieces itself (ranks up to 64 then).  All loads of a wave are on
// their way before the first is waited for; ranks past 64 are loaded as they come.
template <int OUTT, int CT, int COLS, bool JOINED>
__device__ __forceinline__ void up_tile(const AdaptArgs &a, const Tile &t, int rank, int n0, bf16x8 *frag, float *low)
{
    constexpr int NT = UpTerms<OUTT>::N, ESZ = OUTT == OUT_F32 ? 4 : 2;
    const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m = lane & 15, g = lane >> 4;
    const int *rows = rows_of(a);
    const int nb = n0 + wid * 64, n = nb + g * 16, left = a.N - n;
    const __amdgpu_buffer_rsrc_t br = make_rsrc(uniform_ptr(a.b_table[t.e]), (int64_t)a.N * rank * 2);
    int row[CT];
#pragma unroll
    for (int c = 0; c < CT; c++)
        row[c] = rows[t.first + min(c * 16 + m, t.n - 1)];
    auto w_load = [&](int kk, int q) {  // zeros past the rank and past N
        const int col = nb + (m >> 2) * 16 + q * 4 + (m & 3), at = kk * 32 + g * 8;
        return __builtin_bit_cast(bf16x8, bload16(br, at < rank ? (col * rank + at) * 2 : -16, 0));
    };
    auto h_load = [&](int c, int kk, int q) {
        return *(const bf16x8 *)(a.low + ((int64_t)q * a.B + t.first + min(c * 16 + m, t.n - 1)) * a.ldk + kk * 32 + g * 8);
    };
    const int KK = (rank + 31) >> 5;
    bf16x8 w[2][4];
#pragma unroll
    for (int kk = 0; kk < 2; kk++)
#pragma unroll
        for (int q = 0; q < 4; q++)
            w[kk][q] = w_load(kk, q);
    // (row tile, 32 ranks, term) a wave in turn
    constexpr int HN = JOINED ? (CT * 2 * NT + AD_UP - 1) / AD_UP : 1;
    bf16x8 h[HN];
    if constexpr (JOINED) {
#pragma unroll
        for (int j = 0; j < HN; j++) {
            const int i = min(j * AD_UP + wid, CT * 2 * NT - 1);
            h[j] = h_load(i / (2 * NT), min(i / NT % 2, (a.ldk >> 5) - 1), i % NT);
        }
    }
    Out16<OUTT> base[CT];
#pragma unroll
    for (int c = 0; c < CT; c++) {
        const bool ok = row[c] >= 0 && row[c] < a.B;
        const uint8_t *p = (const uint8_t *)a.base + (int64_t)(ok ? row[c] : 0) * a.ldb * ESZ;
        // of a row that is there, whatever the lane: no branch, no wait
        base[c].load(p + (int64_t)(COLS == COLS_ALL ? n : min(n, a.N - 16)) * ESZ);
        if (!ok && c * 16 + m < t.n)
            __hip_atomic_fetch_or(a.status, DEV_BAD_ADAPTER, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (!ok || c * 16 + m >= t.n || left <= 0)
            row[c] = -1;
    }
    if constexpr (JOINED) {
#pragma unroll
        for (int j = 0; j < HN; j++)
            if (j * AD_UP + wid < CT * 2 * NT)
                frag[(j * AD_UP + wid) * 64 + lane] = h[j];
    } else {
        // (row tile, 32 ranks) a wave, or two of them, all loads of both in flight; where
        // there are fewer than waves, several waves share a lane's eight ranks.  The pieces
        // are added in order either way: a row's bits do not depend on how many rows its
        // tile has.
        const int parts = CT * KK;  // a power of two: KK is 1 or 2
        const float f = a.factors ? a.factors[t.e] : 1.f;
        const int64_t step = (int64_t)a.B * a.ldp;
        // past the rank: of ranks that are there, made zeros by terms()
        auto place = [&](int part) {
            const int c = part >> (KK - 1), kk = part & (KK - 1);
            return a.part + (int64_t)(t.first + min(c * 16 + m, t.n - 1)) * a.ldp + min(kk * 32 + g * 8, rank - 8);
        };
        auto terms = [&](int part, float *v) {
            const bool there = (part & (KK - 1)) * 32 + g * 8 < rank;
#pragma unroll
            for (int j = 0; j < 8; j++)
                v[j] = there ? v[j] * f : 0.f;
            const Split<NT> sp = split_f32<NT>(v);
#pragma unroll
            for (int q = 0; q < NT; q++)
                frag[(((part >> (KK - 1)) * 2 + (part & (KK - 1))) * NT + q) * 64 + lane] = sp.t[q];
        };
        if (CT > 2 || parts >= AD_UP) {
            constexpr int PW = CT * 2 > AD_UP ? CT * 2 / AD_UP : 1;
            float v[PW][8];
            const float *p[PW];
#pragma unroll
            for (int w = 0; w < PW; w++) {
                p[w] = place((w * AD_UP + wid) & (parts - 1));
#pragma unroll
                for (int j = 0; j < 8; j++)
                    v[w][j] = 0.f;
            }
#pragma unroll 8
            for (int s = 0; s < a.split; s++)
#pragma unroll
                for (int w = 0; w < PW; w++) {
                    const f32x4 lo = *(const f32x4 *)(p[w] + s * step), hi = *(const f32x4 *)(p[w] + s * step + 4);
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        v[w][j] += lo[j];
                        v[w][4 + j] += hi[j];
                    }
                }
#pragma unroll
            for (int w = 0; w < PW; w++)
                if (w * AD_UP < parts)
                    terms(w * AD_UP + wid, v[w]);
        } else {
            // W of the eight ranks, eight pieces in flight; those past the last are it
            // again, and nothing is added of them
            auto share = [&](auto width) {
                constexpr int W = decltype(width)::value;
                const int part = wid & (parts - 1), at = (wid >> (parts - 1)) * W;
                const float *p = place(part) + at;
                float v[W];
#pragma unroll
                for (int j = 0; j < W; j++)
                    v[j] = 0.f;
                for (int s0 = 0; s0 < a.split; s0 += 8) {
                    uint32_t x[8][W];
#pragma unroll
                    for (int s = 0; s < 8; s++)
                        __builtin_memcpy(x[s], p + min(s0 + s, a.split - 1) * step, 4 * W);
#pragma unroll
                    for (int s = 0; s < 8; s++) {
                        const uint32_t in = s0 + s < a.split ? 0xFFFFFFFFu : 0u;
#pragma unroll
                        for (int j = 0; j < W; j++)
                            v[j] += __uint_as_float(x[s][j] & in);
                    }
                }
                __builtin_memcpy(low + (part * 64 + lane) * 8 + at, v, 4 * W);
            };
            if (parts == 1)
                share(std::integral_constant<int, 2>());
            else
                share(std::integral_constant<int, 4>());
            __syncthreads();
            if (wid < parts) {
                float v[8];
                __builtin_memcpy(v, low + (wid * 64 + lane) * 8, 32);
                terms(wid, v);
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < CT; c++) {
        f32x4 acc[4];
#pragma unroll
        for (int q = 0; q < 4; q++)
            acc[q] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kk = 0; kk < 2; kk++) {
            if (kk == 1 && KK < 2)
                break;
#pragma unroll
            for (int s = 0; s < NT; s++) {
                const bf16x8 hv = frag[((c * 2 + kk) * NT + s) * 64 + lane];
#pragma unroll
                for (int q = 0; q < 4; q++)
                    acc[q] = mfma(w[kk][q], hv, acc[q]);
            }
        }
        if constexpr (JOINED) {
            for (int kk = 2; kk < KK; kk++) {
                bf16x8 wk[4], hk[NT];
#pragma unroll
                for (int q = 0; q < 4; q++)
                    wk[q] = w_load(kk, q);
#pragma unroll
                for (int s = 0; s < NT; s++)
                    hk[s] = h_load(c, kk, s);
#pragma unroll
                for (int s = 0; s < NT; s++)
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        acc[q] = mfma(wk[q], hk[s], acc[q]);
            }
        }
        if constexpr (COLS == COLS_END)
            base[c].move_down(n - min(n, a.N - 16));  // what was loaded ends with the row
        if (row[c] >= 0) {
            float v[16];
#pragma unroll
            for (int q = 0; q < 4; q++)
#pragma unroll
                for (int j = 0; j < 4; j++)
                    v[q * 4 + j] = base[c].at(q * 4 + j) + acc[q][j];
            store16<OUTT>((uint8_t *)a.y + ((int64_t)row[c] * a.ldy + n) * ESZ, COLS == COLS_ALL ? 16 : left, v);
        }
    }
}

template <int OUTT, int COLS, bool JOINED>
__device__ __forceinline__ void up_rows(const AdaptArgs &a, const Tile &t, int rank, int n0, bf16x8 *frag, float *low)
{
    if (t.n <= 16)
        up_tile<OUTT, 1, COLS, JOINED>(a, t, rank, n0, frag, low);
    else if (t.n <= 32)
        up_tile<OUTT, 2, COLS, JOINED>(a, t, rank, n0, frag, low);
    else
        up_tile<OUTT, 4, COLS, JOINED>(a, t, rank, n0, frag, low);
}

// Rows without an adapter: y = base, 64 columns a wave from nb.
template <int OUTT>
__device__ __forceinline__ void copy_tile(const AdaptArgs &a, const Tile &t, int nb)
{
    constexpr int ESZ = OUTT == OUT_F32 ? 4 : 2;
    const int lane = threadIdx.x & 63, n = nb + (lane >> 4) * 16, left = a.N - n;
    for (int i = lane & 15; i < t.n; i += 16) {
        const int row = rows_of(a)[t.first + i];
        if (row < 0 || row >= a.B) {
            __hip_atomic_fetch_or(a.status, DEV_BAD_ADAPTER, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        } else if (left > 0) {
            Out16<OUTT> v;
            const uint8_t *p = (const uint8_t *)a.base + (int64_t)row * a.ldb * ESZ;
            const int at = min(n, a.N - 16);
            v.load(p + (int64_t)at * ESZ);
            v.move_down(n - at);
            float o[16];
#pragma unroll
            for (int j = 0; j < 16; j++)
                o[j] = v.at(j);
            store16<OUTT>((uint8_t *)a.y + ((int64_t)row * a.ldy + n) * ESZ, left, o);
        }
    }
}

// Three waves a SIMD with bf16 outputs, which 142 and 154 registers give without being
// asked; the bound keeps it so (at two, 64 rows of 32 adapters took 10.8 us instead of 8.9).
template <int OUTT, bool JOINED>
__global__ __launch_bounds__(64 * AD_UP, OUTT == OUT_BF16 ? 3 : 2) void adapt_up_kernel(AdaptArgs a, int nchunks)
{
    __shared__ bf16x8 frag[4 * 2 * UpTerms<OUTT>::N * 64];  // 16 or 24 KB
    __shared__ __align__(16) float low[JOINED ? 1 : 2 * 64 * 8];  // 4 KB
    const int n0 = blockIdx.x % nchunks * AD_UP * 64;
    Tile t;
    if (!tile_of(a, blockIdx.x / nchunks, &t, n0 == 0 && threadIdx.x == 0))
        return;
    const int rank = rank_of(a, t.e, n0 == 0 && threadIdx.x == 0);
    if (rank == 0) {
        if (a.base != a.y)  // in place these rows stand
            copy_tile<OUTT>(a, t, n0 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 64);
        return;
    }
    if (n0 + AD_UP * 64 <= a.N)
        up_rows<OUTT, COLS_ALL, JOINED>(a, t, rank, n0, frag, low);
    else
        up_rows<OUTT, COLS_END, JOINED>(a, t, rank, n0, frag, low);
}

// Pieces of K, by B alone: how many adapters the rows name is known on the device
// only.  Every piece is read again by the second product, so pieces are no smaller
// than 768 elements (5120 x 5120, all launches; 16 rows of as many adapters of rank
// 16: 9.3 us at 256, 7.5 at 768, 8.2 at 1536; 64 rows of 32: 13.1, 9.1, 9.9; 64 rows of
// one of rank 64: 22.2, 17.9, 21.8; but 16 rows of K = 17408: 17.6, 11.3, 9.5, 70 in fp32
// 19.0, 13.6, 11.4), and there are fewer of them where the rows make
// enough tiles for the chip (4096 rows of rank 16: 38.3 us at 512, 36.9 at 768, 33.6
// at 1536; 2048 rows of rank 64: 35.4, 31.2, 33.9, and 31.6 at 1024, the choice).
void adapt_shape(AdaptArgs &a)
{
    const int tiles = (a.B + AD_ROWS - 1) / AD_ROWS, pieces = tiles > 192 ? 1 : 192 / tiles;
    const int kc = ((a.K + pieces - 1) / pieces + 255) / 256 * 256;
    a.kc = kc < 768 ? 768 : kc;
    a.split = (a.K + a.kc - 1) / a.kc;
    a.ldp = (a.rank + 15) / 16 * 16;
    a.ldk = (a.rank + 31) / 32 * 32;
}

// Whether a launch between the two products adds the pieces up: many rows, whose up
// workgroups would each add their tile's again (2048 rows, 5120 x 5120 at rank 64:
// 33.7 us without, 31.5 with; 5120 to 17408 at rank 16: 53.2 and 51.8, but 17408 to 5120
// 40.5 and 44.2; 512 rows of eight at rank 16: 15.4 and 17.2, 1000 18.4 and 19.8), and
// ranks that a workgroup does not hold at once.
static bool adapt_joins(int64_t B, int64_t rank) { return rank > AD_CHUNK || B > 1024; }

int64_t adapt_part_bytes(int64_t B, int64_t K, int64_t rank)
{
    AdaptArgs a = {};
    a.B = (int)B;
    a.K = (int)K;
    a.rank = (int)rank;
    adapt_shape(a);
    return (int64_t)a.split * B * a.ldp * 4;
}

int64_t adapt_low_bytes(int64_t B, int64_t rank)
{
    return adapt_joins(B, rank) ? 3 * B * ((rank + 31) / 32 * 32) * 2 : 0;
}

template <int OUTT>
static void up_go(const AdaptArgs &a, bool joins, int64_t tiles, hipStream_t st)
{
    const int nchunks = (a.N + AD_UP * 64 - 1) / (AD_UP * 64);
    const dim3 up((unsigned)(tiles * nchunks)), blk(64 * AD_UP);
    if (joins) {
        hipLaunchKernelGGL(adapt_join_kernel<UpTerms<OUTT>::N>, dim3((unsigned)(tiles * 4)), dim3(128), 0, st, a);
        hipLaunchKernelGGL((adapt_up_kernel<OUTT, true>), up, blk, 0, st, a, nchunks);
    } else {
        hipLaunchKernelGGL((adapt_up_kernel<OUTT, false>), up, blk, 0, st, a, nchunks);
    }
}

hipError_t launch_adapt(int act, int outt, const AdaptArgs &a, hipStream_t st)
{
    const int64_t tiles = adapter_tiles(a.B, a.E);
    const int chunks = (a.rank + AD_CHUNK - 1) / AD_CHUNK;
    const dim3 down((unsigned)(tiles * chunks * a.split)), blk(64 * AD_WAVES);
    if (act == ACT_F32)
        hipLaunchKernelGGL(adapt_down_kernel<ACT_F32>, down, blk, 0, st, a, chunks);
    else if (act == ACT_BF16)
        hipLaunchKernelGGL(adapt_down_kernel<ACT_BF16>, down, blk, 0, st, a, chunks);
    else
        hipLaunchKernelGGL(adapt_down_kernel<ACT_CODES>, down, blk, 0, st, a, chunks);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    const bool joins = adapt_joins(a.B, a.rank);
    if (outt == QGEMM_F32)
        up_go<OUT_F32>(a, joins, tiles, st);
    else
        up_go<OUT_BF16>(a, joins, tiles, st);
    return hipGetLastError();
}

}  // namespace qg
