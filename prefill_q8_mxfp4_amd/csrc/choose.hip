// The choice of experts: a router's logits to the ids and weights that route and
// combine take, and the gradient of the weights.
//
//   p = softmax(l) or sigmoid(l);  the topk experts of largest key, ties to the
//   lowest index;  weights = scale p, or scale p over the sum of the chosen ones.
//
// The key is p + bias, or without a bias the logit itself, in whose order p is.
// With groups only the `keep` groups of E / groups experts whose one or two best
// keys have the largest sum take part.  p + bias is compared in 64 bits, so that
// two keys an fp32 rounding apart come out in their true order, whatever the
// order of the sum in softmax; logits are compared as they are.
//
// A wave a token; a lane holds EPL neighbouring experts, so the lowest lane with
// the largest key holds the lowest index.  A row is read once; the bytes are few,
// the time is a wave's chain of steps: 2048 tokens of 512 fp32 logits take 3.5 us for
// the best one, 5.0 for ten (a maximum over the wave each), 7.7 for ten by sigmoid,
// bias and groups; 8192 tokens, which fill the vector units, 5.6, 8.7 and 15.4.  Of more
// than 512 experts every key is made in 64 bits where there is a bias or sums of scores,
// and 32 experts a lane take 124 bytes of scratch: 2048 tokens, sigmoid, bias and groups,
// top 10, of 1024 experts 17.0, of 2048 36.1 (the best eight logits: 6.8 and 14.9).
#include <type_traits>

#include "layer.h"

namespace qg {

__device__ __forceinline__ uint64_t wave_top(uint64_t v)
{
    const uint32_t hi = wave_top((uint32_t)(v >> 32));
    const uint32_t lo = wave_top((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return (uint64_t)hi << 32 | lo;
}

__device__ __forceinline__ double wave_total(double v)
{
    for (int d = 32; d; d >>= 1)
        v += __shfl_xor(v, d);
    return v;
}

// ---- keys: whole numbers in the order of the values, 0 for one that is never chosen

__device__ __forceinline__ uint32_t key_of(float v)
{
    if (!(v > -__builtin_inff()))  // -inf or NaN
        return 0u;
    const uint32_t b = __float_as_uint(v + 0.f);  // -0 and 0 are the same
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

__device__ __forceinline__ float value_of(uint32_t k)
{
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

__device__ __forceinline__ uint64_t key_of(double v)
{
    if (!(v > -__builtin_inf()))
        return 0ull;
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}

// EPL neighbouring logits of a row of E; -inf behind its end.
template <int DT, int EPL>
__device__ __forceinline__ void load_logits(const void *base, int64_t at, int left, float *v)
{
    if (left >= EPL) {
        if constexpr (DT == OUT_F32) {
            __builtin_memcpy(v, (const float *)base + at, 4 * EPL);
        } else {
            uint16_t h[EPL];
            __builtin_memcpy(h, (const uint16_t *)base + at, 2 * EPL);
#pragma unroll
            for (int i = 0; i < EPL; i++)
                v[i] = __uint_as_float((uint32_t)h[i] << 16);
        }
    } else {  // every load of a place that is there: none waits for another
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            const int64_t j = at + min(i, left - 1);
            v[i] = DT == OUT_F32 ? ((const float *)base)[j]
                                 : __uint_as_float((uint32_t)((const uint16_t *)base)[j] << 16);
        }
#pragma unroll
        for (int i = 0; i < EPL; i++)
            v[i] = i < left ? v[i] : -__builtin_inff();
    }
}

// A lane's part of the weights of a row from its chosen logit (0 where it has
// none); `all` is 1 / sum_e exp(l_e - top) for softmax over all experts.
//   renormalised softmax: exp(l - M) over its sum, M the largest chosen one;
//   renormalised sigmoid: p = exp(l - c) exp(c) / (1 + exp(l)) for l <= 0, whose
//   common factor exp(c), c = min(0, M), drops out: no p underflows.
__device__ __forceinline__ float weight_of(bool has, float l, int score, bool renorm, float top, float all)
{
    if (!renorm) {
        float p;
        if (score == QGEMM_SCORE_SOFTMAX) {
            p = expf(l - top) * all;
        } else {  // from exp(-|l|), which holds what p has below 2^-126 too
            const float e = expf(-fabsf(l));
            p = (l > 0.f ? 1.f : e) / (1.f + e);
        }
        return has ? p : 0.f;
    }
    const uint32_t best = wave_top(has ? key_of(l) : 0u);
    const float M = value_of(best);
    float t;
    if (score == QGEMM_SCORE_SOFTMAX)
        t = expf(l - M);
    else
        t = l > 0.f ? 1.f / (1.f + expf(-l)) : expf(l - fminf(M, 0.f)) / (1.f + expf(l));
    t = has && !(l == -__builtin_inff()) ? t : 0.f;
    const float sum = wave_total(t);
    return has && sum != 0.f ? t / sum : 0.f;  // 0: every chosen logit is -inf
}

// What a lane holds of a row.
template <int EPL>
struct Row {
    float v[EPL], bias[EPL];
    int e0;
    float top;  // the largest logit (softmax with keys or sums of scores)
};

// Whether the lanes of one group make a power of two: they meet by exchanges, others
// in LDS.
__device__ __forceinline__ bool groups_meet(int size, int epl)
{
    const int lanes = size / epl;
    return lanes * epl == size && (lanes & (lanes - 1)) == 0;
}

// x of the lane that CTRL says, of the same sixteen.
template <int CTRL>
__device__ __forceinline__ float of_lane(float x)
{
    return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(x), CTRL, 0xF, 0xF, false));
}

template <int CTRL>
__device__ __forceinline__ double of_lane(double x)
{
    const uint64_t b = (uint64_t)__double_as_longlong(x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)b, CTRL, 0xF, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, false);
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}

// The two largest of the lanes of each group, from those of each lane; lane g gets
// those of group g.
template <typename F>
__device__ __forceinline__ void meet_lanes(int lanes, int groups, F *b1, F *b2)
{
    const int lane = threadIdx.x & 63;
    auto join = [&](F x1, F x2) {
        const F low = x1 > *b1 ? *b1 : x1;
        *b1 = x1 > *b1 ? x1 : *b1;
        *b2 = *b2 > x2 ? *b2 : x2;
        *b2 = *b2 > low ? *b2 : low;
    };
    if (lanes > 1)
        join(of_lane<0xB1>(*b1), of_lane<0xB1>(*b2));  // lane ^ 1
    if (lanes > 2)
        join(of_lane<0x4E>(*b1), of_lane<0x4E>(*b2));  // lane ^ 2
    if (lanes > 4)
        join(of_lane<0x141>(*b1), of_lane<0x141>(*b2));  // the other four of eight, alike by now
    if (lanes > 8)
        join(of_lane<0x140>(*b1), of_lane<0x140>(*b2));  // the other eight of sixteen
    for (int d = 16; d < lanes; d <<= 1)
        join(__shfl_xor(*b1, d), __shfl_xor(*b2, d));
    const int from = lane < groups ? lane * lanes : 0;
    *b1 = __shfl(*b1, from);
    *b2 = __shfl(*b2, from);
}

// The two largest of each group, in lane g those of group g.
template <typename F, int EPL>
__device__ __forceinline__ void group_best(const F *part, int e0, int E, int groups, F *mine, F *o1, F *o2)
{
    const int lane = threadIdx.x & 63, size = E / groups, lanes = size / EPL;
    F b1 = (F)-__builtin_inff(), b2 = b1;
    auto add = [&](F x) {
        b2 = x > b1 ? b1 : x > b2 ? x : b2;
        b1 = x > b1 ? x : b1;
    };
    if (groups_meet(size, EPL)) {
#pragma unroll
        for (int i = 0; i < EPL; i++)
            add(part[i]);
        meet_lanes(lanes, groups, &b1, &b2);
    } else {
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (e0 + i < E)
                mine[e0 + i] = part[i];
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");
        __builtin_amdgcn_wave_barrier();
        if (lane < groups)
            for (int i = 0; i < size; i++)
                add(mine[lane * size + i]);
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");
        __builtin_amdgcn_wave_barrier();  // the place may be used again
    }
    *o1 = b1;
    *o2 = b2;
}

// The groups of largest key (lane g holds group g's), as a mask.
template <typename Key>
__device__ __forceinline__ uint64_t keep_groups(Key of, int groups, int keep)
{
    const int lane = threadIdx.x & 63;
    int rank = 0;
    for (int g = 0; g < groups; g++) {
        Key o = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)of, g);
        if constexpr (sizeof(Key) == 8)
            o |= (Key)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(of >> 32), g) << 32;
        rank += g < lane ? o >= of : o > of;
    }
    return __ballot(lane < groups && rank < keep);
}

template <int EPL, typename Key>
__device__ __forceinline__ void drop_groups(Key *key, int e0, int size, uint64_t kept)
{
    const float per = 1.f / (float)size;
    if (groups_meet(size, EPL)) {  // a lane's experts are of one group
        const int g = (int)(((float)e0 + 0.5f) * per);
        const Key in = (kept >> (g & 63)) & 1 ? ~(Key)0 : (Key)0;
#pragma unroll
        for (int i = 0; i < EPL; i++)
            key[i] &= in;
        return;
    }
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const int g = (int)(((float)(e0 + i) + 0.5f) * per);  // exact: e below 2^11, half a step from any border
        if (!((kept >> (g & 63)) & 1))
            key[i] = 0;
    }
}

// The choice as it is defined: keys in 64 bits (WIDE) or the logits.  Lane j gets the
// j-th expert and its logit.
template <int EPL, bool WIDE>
__device__ __forceinline__ void choose_exactly(const ChooseArgs &a, const Row<EPL> &r, double *lds, int *id, float *l)
{
    typedef typename std::conditional<WIDE, uint64_t, uint32_t>::type Key;
    const int lane = threadIdx.x & 63;
    Key key[EPL];
    double part[WIDE ? EPL : 1];  // p + bias, what a group's key is the sum of
    if constexpr (WIDE) {
        if (a.score == QGEMM_SCORE_SOFTMAX) {
            double s = 0.0;
#pragma unroll
            for (int i = 0; i < EPL; i++) {
                part[i] = exp((double)r.v[i] - (double)r.top);
                s += part[i];
            }
            s = wave_total(s);
#pragma unroll
            for (int i = 0; i < EPL; i++)
                part[i] = part[i] / s;
        } else {
#pragma unroll
            for (int i = 0; i < EPL; i++)
                part[i] = 1.0 / (1.0 + exp(-(double)r.v[i]));
        }
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            part[i] += (double)r.bias[i];
            if (key_of(r.v[i]) == 0u || key_of(part[i]) == 0ull)
                part[i] = -__builtin_inf();
            key[i] = a.bias ? key_of(part[i]) : (uint64_t)key_of(r.v[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < EPL; i++)
            key[i] = key_of(r.v[i]);
    }
    if (a.groups > 1) {
        uint64_t of;
        if constexpr (WIDE) {
            double b1, b2;
            group_best<double, EPL>(part, r.e0, a.E, a.groups, lds, &b1, &b2);
            of = key_of(a.best == 2 ? b1 + b2 : b1);
        } else {
            float v[EPL], b1, b2;
#pragma unroll
            for (int i = 0; i < EPL; i++)
                v[i] = key[i] ? r.v[i] : -__builtin_inff();
            group_best<float, EPL>(v, r.e0, a.E, a.groups, (float *)lds, &b1, &b2);
            of = key_of(b1);
        }
        drop_groups<EPL>(key, r.e0, a.E / a.groups, keep_groups(of, a.groups, a.keep));
    }
    *id = -1;
    *l = 0.f;
    for (int j = 0; j < a.topk; j++) {  // the largest key of the wave
        Key b = 0;
        int bi = 0;
        float bv = 0.f;
#pragma unroll
        for (int i = EPL - 1; i >= 0; i--) {
            const bool up = key[i] >= b;
            b = up ? key[i] : b;
            bi = up ? i : bi;
            bv = up ? r.v[i] : bv;
        }
        const Key best = wave_top(b);
        if (best == 0)
            break;
        const int win = __ffsll((unsigned long long)__ballot(b == best)) - 1;
        const int i_win = __builtin_amdgcn_readlane(bi, win);
        const float v_win = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(bv), win));
        if (lane == j) {
            *id = win * EPL + i_win;
            *l = v_win;
        }
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (lane == win && i == i_win)
                key[i] = 0;
    }
}

// The groups to keep where fp32 does not tell them apart (sigmoid, lanes that meet):
// exact keys of the experts that may be among their group's best, those of `last`
// (lane g: the last of group g's fp32 keys that count) or nearer to it than `off`.
// A lane rarely has more than one, so this is one exponential in 64 bits, not EPL.
template <int EPL>
__device__ __forceinline__ uint64_t keep_exactly(const ChooseArgs &a, const Row<EPL> &r, const float *part, float last,
                                                 float off)
{
    const int lane = threadIdx.x & 63, lanes = a.E / a.groups / EPL;
    const float from = __shfl(last, min(lane / lanes, a.groups - 1)) - off;
    uint32_t need = 0;
#pragma unroll
    for (int i = 0; i < EPL; i++)
        need |= part[i] > -__builtin_inff() && part[i] >= from ? 1u << i : 0u;
    double b1 = -__builtin_inf(), b2 = b1;
    while (__ballot(need != 0)) {
        const int at = __ffs(need) - 1;
        float v = 0.f, bias = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            v = i == at ? r.v[i] : v;
            bias = i == at ? r.bias[i] : bias;
        }
        const double x = need ? 1.0 / (1.0 + exp(-(double)v)) + (double)bias : -__builtin_inf();
        b2 = x > b1 ? b1 : x > b2 ? x : b2;
        b1 = x > b1 ? x : b1;
        need &= need - 1;
    }
    meet_lanes(lanes, a.groups, &b1, &b2);
    return keep_groups(key_of(a.best == 2 ? b1 + b2 : b1), a.groups, a.keep);
}

// The same from fp32 keys, for up to eight experts a lane: their lowest three bits
// give way to the place in the lane, so that a lane sorts its words once and a turn
// is a maximum over the wave and a shift in the lane that had it.  Where the order
// hangs on bits that these keys do not hold (keys of which only the lowest three
// bits tell which is larger; WIDE, keys nearer than `near`, a bound on the errors of
// both), the choice goes on until the next key is clearly smaller, and the exact keys
// of the candidates, one a lane, put them in order.  (Logits in bf16 lose nothing.)
// Returns false where that does not do: groups of softmax scores too near each other,
// more than 64 candidates.
template <int DT, int EPL, bool WIDE>
__device__ __forceinline__ bool choose_fast(const ChooseArgs &a, const Row<EPL> &r, int64_t t, double *lds, int *id,
                                            float *l)
{
    const int lane = threadIdx.x & 63;
    uint32_t key[EPL];
    float near = 0.f;
    if constexpr (WIDE) {
        // The hardware's exponential of x is within (|x| + 4) 2^-24 of itself (its argument
        // is rounded after a product) and its reciprocal within 2^-23.  Sigmoid: p' = p (1 - p)
        // and |x| p (1 - p) < 0.3 leave p within 2^-21.  Softmax: with d = top - l, p d < 0.4
        // pmax, and the sum's 38 roundings leave p within 2^-17 pmax.  p + bias rounds once.
        float part[EPL], pmax = 0.f, kmax = 0.f;
        if (a.score == QGEMM_SCORE_SOFTMAX) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < EPL; i++) {
                part[i] = __expf(r.v[i] - r.top);
                s += part[i];
            }
            s = 1.f / wave_total(s);
#pragma unroll
            for (int i = 0; i < EPL; i++)
                part[i] *= s;
        } else {
#pragma unroll
            for (int i = 0; i < EPL; i++)
                part[i] = __builtin_amdgcn_rcpf(1.f + __expf(-r.v[i]));
        }
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            pmax = fmaxf(pmax, part[i]);
            part[i] += r.bias[i];
            const bool live = r.v[i] > -__builtin_inff() && part[i] > -__builtin_inff();
            part[i] = live ? part[i] : -__builtin_inff();
            kmax = fmaxf(kmax, live ? fabsf(part[i]) : 0.f);
            key[i] = key_of(a.bias ? part[i] : r.v[i]);
        }
        pmax = __uint_as_float(wave_top(__float_as_uint(pmax)));
        kmax = __uint_as_float(wave_top(__float_as_uint(kmax)));
        // both keys' errors; `near` with the three bits of each too (2^-20 of it)
        const float off = 2.f * ((a.score == QGEMM_SCORE_SOFTMAX ? 0x1p-17f * pmax : 0x1p-21f) + 0x1p-24f * kmax);
        near = off + 0x1p-19f * kmax;
        if (a.groups > 1) {
            float b1, b2;
            group_best<float, EPL>(part, r.e0, a.E, a.groups, (float *)lds, &b1, &b2);
            const uint32_t of = key_of(a.best == 2 ? b1 + b2 : b1);
            uint64_t kept = keep_groups(of, a.groups, a.keep);
            const bool in = (kept >> lane) & 1, out = lane < a.groups && !in;
            const uint32_t least = ~wave_top(in ? ~of : 0u), most = wave_top(out ? of : 0u);
            // (differences of -inf and NaN are not apart)
            if (a.keep < a.groups && !(value_of(least) - value_of(most) > 2.f * off + 0x1p-22f * kmax)) {
                if (a.score != QGEMM_SCORE_SIGMOID || !groups_meet(a.E / a.groups, EPL) || !(kmax < 3e38f))
                    return false;
                kept = keep_exactly<EPL>(a, r, part, a.best == 2 ? b2 : b1, off + 0x1p-22f * kmax);
            }
            drop_groups<EPL>(key, r.e0, a.E / a.groups, kept);
        }
    } else {
#pragma unroll
        for (int i = 0; i < EPL; i++)
            key[i] = key_of(r.v[i]);
        if (a.groups > 1) {
            float v[EPL], b1, b2;
#pragma unroll
            for (int i = 0; i < EPL; i++)
                v[i] = key[i] ? r.v[i] : -__builtin_inff();
            group_best<float, EPL>(v, r.e0, a.E, a.groups, (float *)lds, &b1, &b2);
            drop_groups<EPL>(key, r.e0, a.E / a.groups, keep_groups(key_of(b1), a.groups, a.keep));
        }
    }
    // without a bias the keys of the choice are logits, whatever the groups' were
    const bool scores = WIDE && a.bias;
    const bool exact = DT == OUT_BF16 && !scores;
    uint32_t s[8];
#pragma unroll
    for (int i = 0; i < 8; i++)
        s[i] = i < EPL && key[i < EPL ? i : 0] ? (key[i < EPL ? i : 0] & ~7u) | (7 - i) : 0u;
    auto order = [&](int x, int y) {
        const uint32_t hi = max(s[x], s[y]);
        s[y] = min(s[x], s[y]);
        s[x] = hi;
    };
    if constexpr (EPL >= 2) {  // Batcher's network
        order(0, 1);
        if constexpr (EPL >= 4) {
            order(2, 3);
            order(0, 2); order(1, 3);
            order(1, 2);
        }
        if constexpr (EPL == 8) {
            order(4, 5); order(6, 7);
            order(4, 6); order(5, 7);
            order(5, 6);
            order(0, 4); order(1, 5); order(2, 6); order(3, 7);
            order(2, 4); order(3, 5);
            order(1, 2); order(3, 4); order(5, 6);
        }
    }
    // Lane j gets the j-th largest key and its expert; the turns have no branches (eight of
    // them a turn, for what is asked after it now, took as long as the maximum).
    *id = -1;
    *l = 0.f;
    uint32_t mine = 0;
    auto take = [&](int j, uint32_t best) {
        const int win = __ffsll((unsigned long long)__ballot((s[0] & ~7u) == best)) - 1;
        const int i_win = 7 - (__builtin_amdgcn_readlane((int)s[0], win) & 7);
        *id = lane == j ? win * EPL + i_win : *id;
        mine = lane == j ? best : mine;
        if (lane == win) {
#pragma unroll
            for (int i = 0; i < EPL - 1; i++)
                s[i] = s[i + 1];
            s[EPL - 1] = 0u;
        }
    };
    uint32_t best = 0;
    for (int j = 0; j < a.topk; j++) {
        best = wave_top(s[0]) & ~7u;
        take(j, best);
    }
    *id = mine ? *id : -1;  // no key was left
    int count = __popcll(__ballot(mine != 0));
    bool order_it = false;  // some two neighbours are not clearly apart
    if (!exact) {
        auto apart = [&](uint32_t hi, uint32_t lo) { return scores ? value_of(hi) - value_of(lo) > near : lo != hi; };
        const uint32_t before = (uint32_t)__shfl_up((int)mine, 1);
        order_it = __ballot(lane > 0 && mine != 0 && !apart(before, mine)) != 0;
        for (;;) {  // those not clearly smaller than the last
            const uint32_t next = wave_top(s[0]) & ~7u;
            if (next == 0 || apart(best, next))
                break;
            if (count == 64)
                return false;
            order_it = true;
            take(count++, next);
            best = next;
        }
    }
    if (*id >= 0) {  // its logit: the row is in the nearest cache
        float one[1];
        load_logits<DT, 1>(a.logits, t * a.E + *id, 1, one);
        *l = one[0];
    }
    if (order_it) {
        uint64_t k = key_of(*l);
        if (WIDE && a.bias) {
            double p;
            if (a.score == QGEMM_SCORE_SOFTMAX) {
                double sum = 0.0;
#pragma unroll
                for (int i = 0; i < EPL; i++)
                    sum += exp((double)r.v[i] - (double)r.top);
                p = exp((double)*l - (double)r.top) / wave_total(sum);
            } else {
                p = 1.0 / (1.0 + exp(-(double)*l));
            }
            k = key_of(p + (double)(lane < count ? a.bias[*id] : 0.f));
        }
        int rank = lane;
        if (lane < count)
            rank = 0;
        for (int g = 0; g < count; g++) {
            const uint64_t o = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)k, g) |
                               (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(k >> 32), g) << 32;
            const int oid = __builtin_amdgcn_readlane(*id, g);
            if (lane < count)
                rank += o > k || (o == k && oid < *id);
        }
        // every lane sends to another one: ranks below count, the rest to itself
        *id = __builtin_amdgcn_ds_permute(rank * 4, *id);
        *l = __uint_as_float((uint32_t)__builtin_amdgcn_ds_permute(rank * 4, (int)__float_as_uint(*l)));
    }
    if (lane >= a.topk) {  // candidates past the choice
        *id = -1;
        *l = 0.f;
    }
    return true;
}

template <int DT, int EPL, bool WIDE>
__global__ __launch_bounds__(256) void choose_kernel(ChooseArgs a)
{
    extern __shared__ double group_lds[];
    const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 6) + wid;
    if (t >= a.T)
        return;
    double *mine = group_lds + (size_t)wid * a.E;
    Row<EPL> r;
    r.e0 = lane * EPL;
    load_logits<DT, EPL>(a.logits, t * a.E + r.e0, a.E - r.e0, r.v);
    if (WIDE) {
#pragma unroll
        for (int i = 0; i < EPL; i++)
            r.bias[i] = 0.f;
        if (a.bias)
            load_logits<OUT_F32, EPL>(a.bias, r.e0, a.E - r.e0, r.bias);
    }
    bool odd = false;  // a NaN, or an infinity that softmax makes one
    float top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        odd |= r.v[i] != r.v[i];
        top = fmaxf(top, r.v[i]);  // of a NaN and a number the number
    }
    const bool bad = __ballot(odd || (a.score == QGEMM_SCORE_SOFTMAX && top == __builtin_inff())) != 0;
    // the largest logit and the sum over all experts, where softmax asks for them
    float all = 0.f;
    r.top = 0.f;
    const bool whole = a.score == QGEMM_SCORE_SOFTMAX && (WIDE || !a.renorm);
    if (whole)
        r.top = value_of(wave_top(key_of(top)));
    if (whole && !a.renorm) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; i++)
            s += expf(r.v[i] - r.top);
        all = 1.f / wave_total(s);
    }
    int id = -1;
    float l = 0.f;
    bool sure = false;
    if constexpr (EPL <= 8)
        sure = choose_fast<DT, EPL, WIDE>(a, r, t, mine, &id, &l);
    if (!sure)
        choose_exactly<EPL, WIDE>(a, r, mine, &id, &l);
    const float w = a.scale * weight_of(id >= 0, l, a.score, a.renorm, r.top, all);
    if (lane < a.topk) {
        a.ids[t * a.topk + lane] = id;
        a.weights[t * a.topk + lane] = bad ? __builtin_nanf("") : w;
    }
}

// dl from dw, the ids constant; with g_j = scale dw_j, w_j the weights over scale
// and sums over the row's choices:
//   renormalised softmax:  d_j = w_j (g_j - sum g w)          on the chosen
//   renormalised sigmoid:  d_j = (1 - p_j) w_j (g_j - sum g w)   "
//   sigmoid:               d_j = g_j p_j (1 - p_j)               "
//   softmax:               dl_e = p_e (sum_{j: id_j = e} g_j - sum g p)
template <int DT, int EPL>
__global__ __launch_bounds__(256) void choose_grad_kernel(ChooseGradArgs a)
{
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 6) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (t >= a.T)
        return;
    const int e0 = lane * EPL;
    const bool dense = a.score == QGEMM_SCORE_SOFTMAX && !a.renorm;
    int id = lane < a.topk ? a.ids[t * a.topk + lane] : -1;
    const bool has = id >= 0 && id < a.E;
    float l = 0.f, g = 0.f;
    if (has) {
        float one[1];
        load_logits<DT, 1>(a.logits, t * a.E + id, 1, one);
        l = one[0];
        g = a.scale * a.dweights[t * a.topk + lane];
    }
    id = has ? id : -1;
    float p[EPL], d[EPL];
    float top = 0.f, all = 0.f;
    if (dense) {
        load_logits<DT, EPL>(a.logits, t * a.E + e0, a.E - e0, p);
        uint32_t most = 0;
        bool odd = false;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            most = max(most, key_of(p[i]));
            odd |= p[i] != p[i];
        }
        const uint32_t k = wave_top(most);
        // a row of -inf has no weights and no gradient, one with a NaN NaNs
        top = __ballot(odd) != 0 ? __builtin_nanf("") : k ? value_of(k) : 0.f;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            p[i] = expf(p[i] - top);
            s += p[i];
        }
        s = wave_total(s);
        all = s == 0.f ? 0.f : 1.f / s;
    }
    const float w = weight_of(has, l, a.score, a.renorm, top, all);
    float val = g;
    float dot = 0.f;
    if (a.renorm || dense)
        dot = wave_total(has ? g * w : 0.f);
    if (a.renorm)
        val = w * (g - dot);
    if (a.score == QGEMM_SCORE_SIGMOID) {
        const float e = expf(-fabsf(l)), rest = (l > 0.f ? e : 1.f) / (1.f + e);  // 1 - p
        val = a.renorm ? val * rest : g * w * rest;
    }
#pragma unroll
    for (int i = 0; i < EPL; i++)
        d[i] = 0.f;
    for (int j = 0; j < a.topk; j++) {
        const int at = __builtin_amdgcn_readlane(id, j) - e0;
        const float x = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(val), j));
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (at == i)
                d[i] += x;
    }
    if (dense) {
#pragma unroll
        for (int i = 0; i < EPL; i++)
            d[i] = p[i] * all * (d[i] - dot);
    }
    const int left = a.E - e0;
    const int64_t to = t * a.E + e0;
    if (left >= EPL) {
        if constexpr (DT == OUT_F32) {
            __builtin_memcpy((float *)a.dlogits + to, d, 4 * EPL);
        } else {
            __bf16 h[EPL];
#pragma unroll
            for (int i = 0; i < EPL; i++)
                h[i] = (__bf16)d[i];
            __builtin_memcpy((__bf16 *)a.dlogits + to, h, 2 * EPL);
        }
    } else {
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (i < left)
                store_out<DT>(a.dlogits, to + i, d[i]);
    }
}

// Waves a workgroup: one while the tokens are few, so that they spread over the
// chip.  Of many tokens fewer, larger workgroups start a little sooner (ten of softmax,
// 8192 tokens: 9.1 us with one wave, 8.9 with two, 8.7 with four).
static int waves_of(int64_t T) { return T <= 1024 ? 1 : 4; }

template <int DT, int EPL>
static hipError_t choose_go(const ChooseArgs &a, hipStream_t st)
{
    const int W = waves_of(a.T);
    const dim3 grid((unsigned)((a.T + W - 1) / W)), blk(64 * W);
    const bool wide = a.bias || (a.groups > 1 && a.best == 2);
    const int lds = a.groups > 1 ? W * a.E * 8 : 0;  // 64 KB at most
    if (wide)
        hipLaunchKernelGGL((choose_kernel<DT, EPL, true>), grid, blk, lds, st, a);
    else
        hipLaunchKernelGGL((choose_kernel<DT, EPL, false>), grid, blk, lds, st, a);
    return hipGetLastError();
}

template <int DT, int EPL>
static hipError_t choose_grad_go(const ChooseGradArgs &a, hipStream_t st)
{
    const int W = waves_of(a.T);
    hipLaunchKernelGGL((choose_grad_kernel<DT, EPL>), dim3((unsigned)((a.T + W - 1) / W)), dim3(64 * W), 0, st, a);
    return hipGetLastError();
}

#define QG_BY_EPL(go, DT)                                   \
    do {                                                    \
        if (a.E <= 64) return go<DT, 1>(a, st);             \
        if (a.E <= 128) return go<DT, 2>(a, st);            \
        if (a.E <= 256) return go<DT, 4>(a, st);            \
        if (a.E <= 512) return go<DT, 8>(a, st);            \
        if (a.E <= 1024) return go<DT, 16>(a, st);          \
        return go<DT, 32>(a, st);                           \
    } while (0)

hipError_t launch_choose(int dt, const ChooseArgs &a, hipStream_t st)
{
    if (dt == QGEMM_F32)
        QG_BY_EPL(choose_go, OUT_F32);
    QG_BY_EPL(choose_go, OUT_BF16);
}

hipError_t launch_choose_grad(int dt, const ChooseGradArgs &a, hipStream_t st)
{
    if (dt == QGEMM_F32)
        QG_BY_EPL(choose_grad_go, OUT_F32);
    QG_BY_EPL(choose_grad_go, OUT_BF16);
}

}  // namespace qg
