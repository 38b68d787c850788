// distill.cu -- distillation of a student's logit rows from the teacher's top
// logits: the loss of a row, its gradient, or both in one launch.
//
// With q = softmax(s / T) over the student's row s and p the teacher's
// probabilities of the listed ids (softmax(t / T) over the list, or
// exp(t / T - lse_t) with p_rest = 1 - sum p for every other token together):
//   loss   = w [ sum_j p_j (ln p_j - ln q_{id_j}) + p_rest (ln p_rest - ln q_rest) ]
//   dl/ds_v = w / T (q_v - p_v)                  v listed (p_v: all its entries)
//   dl/ds_v = w / T q_v (1 - p_rest / q_rest)    otherwise (p_rest = 0: w / T q_v)
//
// Everything the gradient needs of a row is its maximum, 1 / sum, the share of all
// but the largest listed token, reference and factor of the tokens that are not
// listed, and the list: `state` holds it between the two calls.
//
// All three are bound by HBM: the loss by one read of the row, the gradient by a
// read and a write.
//  * distill_stream_kernel streams a row through registers for its loss.
//    512 rows of 126464 bf16 tokens, 64 teacher logits: 38 us with an empty L2
//    (3.4 TB/s of 6.8; 3.4 CTAs per SM, each with 16 KB on its way).  Two CTAs
//    per row took 46 us.
//  * The step needs the row twice, once for its sums and once for the gradient:
//    distill_row_kernel holds it on chip in between.  A cluster's CTAs copy a
//    slice each (about 40 KB, five CTAs per SM) into shared memory with
//    asynchronous copies, read the teacher's list while those are on their way,
//    add up their slice, exchange sums through distributed shared memory and
//    write their slice's gradient.  The gradient alone is the same without the
//    sums.  How long a CTA lives decides (its slice takes its share of the SM's
//    shared memory meanwhile), so its reductions share five barriers, only the
//    first CTA does 64-bit arithmetic on the sums, and last.
//    2048 rows of 152064 bf16 tokens, a quarter of them without a loss: 224 us,
//    4.9 TB/s of the 1.09 GB that it reads and writes (a call among others).
//    Registers decide here: at 48 of them, with what only the loss needs at the
//    end kept in shared memory, nothing spills; with 92 bytes of spills it took
//    255 us.  Against 228 us then, streamed twice (the second read from L2) it took
//    269 us at best, slices of 77 KB 308 us, 128 threads 231 us.
//  * Rows that eight CTAs can not hold (above 1.5 MB) are streamed twice.
//
// q_rest = 1 - sum q_id would lose all digits for a peaked student, so the sum
// over the tokens that are not listed is taken apart from the start: listed
// logits are taken out (-inf in their place), by the row kernel in its slice, by
// the stream kernel with a bitmap, one byte of which answers for a whole vector.
// The gradient is written for every token as if none were listed, and then the
// listed ones are written over (the block barrier between orders the two).
#include "common.cuh"
#include "launch.h"
#include "row_vec.cuh"
#include "weight.cuh"

namespace dlm {

namespace {

constexpr int kThreads = kRowThreads;
constexpr int kWarps = kRowWarps;
constexpr int kUnroll = 4;
constexpr float kRebase = 12.0f;  // powers of 2 of headroom before a thread's reference moves

// What a thread, a warp or a CTA knows of a row: the softmax sums of its slice over
// the listed tokens, relative to the largest of them `ref` (-inf: none), and over
// the others, relative to `rest_ref` (a NaN logit makes its reference NaN).  Two references,
// since a student's list may lie far above the rest: with one, the rest's weights
// were subnormal or 0 from 83 nats on, and the quotients that p_rest is multiplied
// by overflowed.  `listed` leaves one weight of 1, that of a token at `ref`, out: a
// student that is sure of a token has 1 - q from the others' sum, which 1 + that
// sum would have rounded away (and the gradient there is (1 - p) - (1 - q)).  Its
// sign says whether an id may be listed twice.
// (16 bytes: one store into another CTA, one load.)
struct __align__(16) Share {
    float ref, listed, rest_ref, rest;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(DLM_FULL_MASK, v, o);
    return v;
}

__device__ __forceinline__ float or_zero(float ref) { return ref > -INFINITY ? ref : 0.f; }
__device__ __forceinline__ bool is_twice(float listed) { return __float_as_uint(listed) >> 31; }

// A sum that is relative to `ref` relative to `to` (-inf: nothing, and 0).
__device__ __forceinline__ float rebased(float sum, float ref, float to, float c) {
    return sum * ex2((ref - or_zero(to)) * c);
}

// The sum over the lanes in a fixed order, all lanes get it: common references
// first, then plain sums.
__device__ __forceinline__ Share warp_share(Share a, float c) {
    Share b;
    b.ref = warp_max_nan(a.ref);
    b.rest_ref = warp_max_nan(a.rest_ref);
    const bool twice = __any_sync(DLM_FULL_MASK, is_twice(a.listed));
    // the first lane at the common reference leaves its 1 out for all
    const bool first = (threadIdx.x & 31) == __ffs(__ballot_sync(DLM_FULL_MASK, a.ref == b.ref)) - 1;
    b.listed = warp_sum(rebased(fabsf(a.listed) + (first ? 0.f : 1.f), a.ref, b.ref, c));
    b.rest = warp_sum(rebased(a.rest, a.rest_ref, b.rest_ref, c));
    if (twice) b.listed = -b.listed;
    return b;
}

__device__ __forceinline__ Share no_share() { return Share{-INFINITY, 0.f, -INFINITY, 0.f}; }

// What is known of a whole row: its maximum, the sum of all weights relative to
// that, `away` the share of all but one listed token that is at the maximum (-1:
// none is), and the others' sum relative to its own reference, whose weight
// relative to the maximum is `up`.
struct Total {
    float mx, all, away, rest_ref, rest, up;
};

struct Shared {
    Share part[8 * kWarps];   // every warp's of every CTA of the cluster
    float list_max[kWarps];
    uint64_t list_sum[kWarps];
    int flags[kWarps];        // kAny, kBad
    float sum[kWarps];
    uint64_t listed[kWarps];
    Total row;                // row kernel: kept for the loss, which comes last
    float weight, lse_t;
};
enum : int { kAny = 1, kBad = 2 };  // an entry; a teacher logit is NaN or +inf

// The list in shared memory.
struct List {
    int32_t* id;     // -1: no entry
    float* t;        // teacher logit
    float* p;        // teacher weight, not normalised
    float* s;        // student logit (entries of this CTA's slice; the first CTA has all of them)
    uint32_t* own;   // row kernel: this entry took its token out of the slice
    uint32_t* bits;  // stream kernel: the listed tokens of this CTA's slice
};

__host__ __device__ inline size_t shared_bytes() { return (sizeof(Shared) + 15) & ~(size_t)15; }

__device__ __forceinline__ List carve(unsigned char* p, int k) {
    List l;
    p += shared_bytes();
    l.id = reinterpret_cast<int32_t*>(p);
    l.t = reinterpret_cast<float*>(l.id + k);
    l.p = l.t + k;
    l.s = l.p + k;
    l.own = l.bits = reinterpret_cast<uint32_t*>(l.s + k);
    return l;
}

// Bytes of shared memory before a slice.
__host__ __device__ inline size_t slice_offset(int k) { return (shared_bytes() + (size_t)k * 20 + 15) & ~(size_t)15; }

__device__ __forceinline__ float teacher_at(const DistillArgs& a, int64_t i) {
    switch (a.teacher_dtype) {
    case DLM_BF16: return Row<DLM_BF16>::scalar(a.teacher, i);
    case DLM_F16: return Row<DLM_F16>::scalar(a.teacher, i);
    default: return static_cast<const float*>(a.teacher)[i];
    }
}

// The list in two steps with a barrier after each.  First: entries into shared
// memory, their maximum per warp.  A thread's first entry may have been asked
// for before (id0, x0).
__device__ __forceinline__ void list_load(const DistillArgs& a, const List& l, Shared& sh, int64_t r, float lse_t,
                                          int id0, float x0) {
    float mx = -INFINITY;
    int flags = fabsf(lse_t) < INFINITY ? 0 : kBad;
    for (int j = threadIdx.x; j < a.k; j += kThreads) {
        const bool first = j < kThreads;
        int id = first ? id0 : a.ids[r * a.k + j];
        const float x = first ? x0 : teacher_at(a, r * a.k + j);
        if (id >= a.vocab) {
            id = -1;
            raise_status(a.dev_status, DLM_DEV_BAD_INDEX);
        }
        if (id >= 0) {
            flags |= x < INFINITY ? (x > -INFINITY ? kAny : 0) : kBad;
            mx = fmaxf(mx, x);
        }
        l.id[j] = id < 0 ? -1 : id;
        l.t[j] = x;
    }
    mx = warp_max_nan(mx);
    flags = __reduce_or_sync(DLM_FULL_MASK, flags);
    if ((threadIdx.x & 31) == 0) {
        sh.list_max[threadIdx.x >> 5] = mx;
        sh.flags[threadIdx.x >> 5] = flags;
    }
}

// Second: the teacher's weights, 2^-(y + lo) each, relative to the list's
// maximum or (rest) to the teacher's log-sum-exp.  The integer weight serves the
// sum, which p_rest is the difference of 1 and; the float keeps all its digits
// for a small one.
__device__ __forceinline__ float list_max(const Shared& sh) {
    float mx = sh.list_max[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, sh.list_max[w]);
    return mx;
}
__device__ __forceinline__ WeightScale teacher_scale(const DistillArgs& a, const Shared& sh) {
    return WeightScale{or_zero(list_max(sh)), a.scale, a.scale_lo, kPow2Neg};
}
// A probability may be above 1 where lse_t lies below the logit (rounded, or
// another row's): up to 2^8, so that the sum of a list fits 64 bits.
constexpr double kMostP = 8 * 0.6931471805599453;
// ln p - ln q of entry j; shift is the student's log-sum-exp less the teacher's.
__device__ __forceinline__ double log_ratio(const DistillArgs& a, const List& l, int j, double shift, bool rest, double lse_s) {
    if (rest && l.p[j] >= 256.f) return kMostP - ((double)l.s[j] * a.inv_t - lse_s);
    return ((double)l.t[j] - (double)l.s[j]) * a.inv_t + shift;
}
// 1 - e^-d for |d| < 2^-12.
__device__ __forceinline__ double one_less_exp(double d) { return d * (1.0 - d * (0.5 - d * (1.0 / 6))); }
// One entry's weight 2^-(y + lo) as an integer.
__device__ __forceinline__ uint64_t teacher_weight(const DistillArgs& a, float x, const WeightScale& ws, bool rest,
                                                   float lse_t, float& y, float& lo) {
    if (!rest) {
        y = weight_exponent(x, ws, lo);
        return weight44_of(y, lo);
    }
    const double d = fmax(-kMostP, (double)lse_t - (double)x * a.inv_t);
    // a teacher that is sure of a token: 1 - p by its series, to the last place (the
    // table's weight is off by 2^-37 of p, 2^-20 of a 1 - p of 10^-5)
    if (fabs(d) < 0x1p-12) {
        y = lo = 0.f;
        return (1ull << kWeightBits) - (uint64_t)__double2ll_rn(one_less_exp(d) * 17592186044416.0);
    }
    const int up = d < 0.0 ? 8 : 0;
    const double e = d * 1.4426950408889634 + up;
    y = (float)e;
    lo = y < INFINITY ? (float)(e - (double)y) : 0.f;
    return weight44_of(fmaxf(y, 0.f), lo) << up;
}
__device__ __forceinline__ void list_weigh(const DistillArgs& a, const List& l, Shared& sh, bool rest, float lse_t) {
    const WeightScale ws = teacher_scale(a, sh);
    uint64_t sum = 0;
    for (int j = threadIdx.x; j < a.k; j += kThreads) {
        float p = 0.f;
        if (l.id[j] >= 0) {
            float y, lo;
            const uint64_t w = teacher_weight(a, l.t[j], ws, rest, lse_t, y, lo);
            sum += w;
            p = y < 16.f ? (float)w * kUnit : y < INFINITY ? exp2f(-y) * fmaf(lo, -kLn2, 1.0f) : 0.f;
        }
        l.p[j] = p;
    }
    sum = (uint64_t)warp_sum_ll((long long)sum);
    if ((threadIdx.x & 31) == 0) sh.list_sum[threadIdx.x >> 5] = sum;
}

// What follows from the list as a whole (after the second barrier).
struct Teacher {
    uint64_t sum;    // of the weights, in 2^-44
    float inv;       // 1 / sum, or 1 when the rest is a class: weight to probability
    float p_rest;
    bool any, bad;
};
__device__ __forceinline__ Teacher list_total(const Shared& sh, bool rest) {
    Teacher t;
    t.sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) t.sum += sh.list_sum[w];
    const uint64_t one = 1ull << kWeightBits;
    t.inv = rest ? 1.f : t.sum ? 1.0f / ((float)t.sum * kUnit) : 0.f;
    t.p_rest = rest && t.sum < one ? (float)(one - t.sum) * kUnit : 0.f;
    int flags = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) flags |= sh.flags[w];
    t.any = flags & kAny;
    t.bad = flags & kBad;
    return t;
}

// The entries that a thread of the stream kernel looks after, j = t, t + kThreads, ...:
// those in the CTA's slice, and of them the first of each token.
constexpr int kMine = (DLM_MAX_TOPK + kThreads - 1) / kThreads;
struct Mine {
    uint32_t in, own;  // a bit per entry
    float s[kMine];    // their logits
};

// The listed tokens of a slice [e0, e1) in its bitmap (zeroed before).
__device__ __forceinline__ void mark_listed(const List& l, int K, int64_t e0, int64_t e1, Mine& mine) {
    mine.in = mine.own = 0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int j = threadIdx.x + i * kThreads;
        const int64_t id = j < K ? l.id[j] : -1;
        if (id < e0 || id >= e1) continue;
        const uint32_t bit = 1u << ((id - e0) & 31);
        mine.in |= 1u << i;
        mine.own |= (uint32_t)((atomicOr(&l.bits[(id - e0) >> 5], bit) & bit) == 0) << i;
    }
}

// Which entry of a token that is listed again marked it first goes by chance, and the
// sums' last place by which thread holds it: the lowest entry has it.
__device__ __forceinline__ void lowest_own(const List& l, int K, Mine& mine) {
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        if (!((mine.in >> i) & 1u)) continue;
        const int j = threadIdx.x + i * kThreads;
        int at = 0;
        while (l.id[at] != l.id[j]) ++at;
        mine.own = (mine.own & ~(1u << i)) | (uint32_t)(at == j) << i;
    }
}

// A vector without the elements of the mask: -inf in their place.
template <int DT>
__device__ __forceinline__ uint4 without(uint4 w, uint32_t mask) {
    uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == DLM_F32) {
            if ((mask >> i) & 1u) x[i] = 0xff800000u;
        } else {
            if ((mask >> (2 * i)) & 1u) x[i] = (x[i] & 0xffff0000u) | Row<DT>::kNegInf;
            if ((mask >> (2 * i + 1)) & 1u) x[i] = (x[i] & 0xffffu) | (uint32_t)Row<DT>::kNegInf << 16;
        }
    }
    return make_uint4(x[0], x[1], x[2], x[3]);
}

// p (x - 1 + e^-x) for x = ln p - ln q, q = p e^-x.  (x of a token at the lowest float
// may pass a float's range where p x does not.)
__device__ __forceinline__ float class_term(float p, double x64, float q) {
    if (!(p > 0.f)) return q;
    const float x = (float)x64;
    if (!(fabsf(x) < INFINITY)) return (float)((double)p * x64);
    if (!(fabsf(x) < 1.f)) return p * (x - 1.f) + q;
    // x^2 (1/2! - x/3! + x^2/4! - ...)
    float r = 1.f / 39916800;
    r = fmaf(-x, r, 1.f / 3628800);
    r = fmaf(-x, r, 1.f / 362880);
    r = fmaf(-x, r, 1.f / 40320);
    r = fmaf(-x, r, 1.f / 5040);
    r = fmaf(-x, r, 1.f / 720);
    r = fmaf(-x, r, 1.f / 120);
    r = fmaf(-x, r, 1.f / 24);
    r = fmaf(-x, r, 1.f / 6);
    r = fmaf(-x, r, 0.5f);
    return p * (x * x * r);
}

// The row's loss, by the first CTA, which has all of the list's student logits;
// q relative to the row's maximum.  sum p x over the classes, x = ln p - ln q,
// loses its digits when student and teacher are near (every x is small, of
// either sign, and off by the log-sum-exps' rounding): with q = p e^-x it is
// sum p (x - 1 + e^-x) + sum p - sum q, whose terms are positive and of second
// order in x, and sum p - sum q is known exactly: 0 with the rest as a class,
// q_rest without.  For that the listed part of q's sum is added up once more,
// from integer weights.  (A list with repeats counts its q twice; it takes the
// plain sum, in 64 bits over the lanes: by one thread it took 30 us for 256
// entries.)  A list of up to kAlone entries is one warp's work:
// `threads` is 32 then, and only warp 0 calls.  Thread 0 has the result.
constexpr int kAlone = 128;

__device__ float row_loss(const DistillArgs& a, const List& l, Shared& sh, const Teacher& tch, Total q,
                          bool rest, float lse_t, bool twice, int threads) {
    const int t = threadIdx.x;
    const WeightScale ws{q.mx, a.scale, a.scale_lo, kPow2Neg};
    if (!twice) {
        uint64_t listed = 0;
        for (int j = t; j < a.k; j += threads)
            if (l.id[j] >= 0) listed += weight44(l.s[j], ws);
        listed = (uint64_t)warp_sum_ll((long long)listed);
        if (threads > 32) {
            if ((t & 31) == 0) sh.listed[t >> 5] = listed;
            __syncthreads();
            listed = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) listed += sh.listed[w];
        }
        q.all = (float)listed * kUnit + q.rest * q.up;
    }
    const double log_all = log_exact(q.all), lse_s = (double)q.mx * a.inv_t + log_all;
    const double log_z = rest ? (double)lse_t
                              : (double)list_max(sh) * a.inv_t + log_exact(fmaxf((float)tch.sum * kUnit, 1.f));
    const double shift = lse_s - log_z;
    // ln p_rest - ln q_rest, from three logarithms: a quotient of the sums has no limit
    const float q_rest = q.rest * q.up / q.all;
    double x_rest = 0;
    if (tch.p_rest > 0.f)
        x_rest = q.rest > 0.f ? log_exact(tch.p_rest) + log_all - log_exact(q.rest) +
                                    ((double)q.mx - (double)q.rest_ref) * a.inv_t
                              : (double)INFINITY;
    if (twice) {
        double v = 0;
        for (int j = t; j < a.k; j += threads)
            if (l.id[j] >= 0 && l.p[j] > 0.f)
                v += (double)(l.p[j] * tch.inv) * log_ratio(a, l, j, shift, rest, lse_s);
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(DLM_FULL_MASK, v, o);
        if (threads > 32) {
            if ((t & 31) == 0) sh.listed[t >> 5] = (uint64_t)__double_as_longlong(v);
            __syncthreads();
            v = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += __longlong_as_double((long long)sh.listed[w]);
        }
        if (tch.p_rest > 0.f) v += (double)tch.p_rest * x_rest;
        return (float)v;
    }
    float v = 0.f;
    const float inv_q = 1.f / q.all;
    for (int j = t; j < a.k; j += threads) {
        if (l.id[j] < 0) continue;
        const double x = log_ratio(a, l, j, shift, rest, lse_s);
        v += class_term(l.p[j] * tch.inv, x, inv_q * exp2f((l.s[j] - q.mx) * a.scale));
    }
    v = warp_sum(v);
    if (threads > 32) {
        if ((t & 31) == 0) sh.sum[t >> 5] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += sh.sum[w];
    }
    if (!rest) return v + q_rest;
    const uint64_t one = 1ull << kWeightBits;
    return v + class_term(tch.p_rest, x_rest, q_rest) + (tch.sum > one ? (float)(tch.sum - one) * kUnit : 0.f);
}

__device__ __forceinline__ void write_state(float* state, const Total& row, float inv, float base, float tail,
                                            float lse_t, bool rest) {
    if (!state) return;
    state[0] = row.mx;
    state[1] = inv;
    state[2] = tail;
    state[3] = lse_t;
    state[4] = rest ? 1.f : 0.f;
    state[5] = base;
    state[6] = row.away;
    state[7] = 0.f;
}

// What the gradient needs of a row: 1 / sum (0: no gradient), and of the tokens
// that are not listed a reference and the factor of their weights relative to it,
// q_v - p_v = tail 2^((z - base) c).
__device__ __forceinline__ bool row_fine(const Teacher& tch, const Total& q) {
    return q.mx > -INFINITY && q.mx < INFINITY && !tch.bad;
}
__device__ __forceinline__ void row_factors(const Teacher& tch, const Total& q, bool rest, float& inv, float& base,
                                            float& tail) {
    inv = rest || tch.any ? 1.f / q.all : 0.f;
    base = q.mx;
    tail = inv;
    if (rest) {
        tail = 0.f;
        if (q.rest > 0.f) {
            base = q.rest_ref;
            tail = inv * q.up - tch.p_rest / q.rest;
        }
    }
    if (!row_fine(tch, q)) inv = tail = NAN;
}

// The loss of a row (the first CTA).
__device__ __forceinline__ void finish_loss(const DistillArgs& a, const List& l, Shared& sh, const Teacher& tch, int64_t r,
                                            float weight, const Total& row, bool rest, float lse_t, bool twice) {
    const bool alone = a.k <= kAlone, fine = row_fine(tch, row);
    if (alone && threadIdx.x >= 32) return;
    float v = NAN;
    if (fine) v = rest || tch.any ? weight * row_loss(a, l, sh, tch, row, rest, lse_t, twice, alone ? 32 : kThreads) : 0.f;
    if (threadIdx.x != 0) return;
    a.loss[r] = v;
    if (!fine) raise_status(a.dev_status, DLM_DEV_NONFINITE);
}

// 2^((z - ref) c) with c in two floats (one float's rounding, the same for every
// token, would show in the loss's seventh digit).
__device__ __forceinline__ f2 weights_of(f2 z, f2 ref, f2 c, f2 c_lo) {
    const f2 d = sub2(z, ref);
    return ex2x2(fma2(d, c, mul2(d, c_lo)));  // the large product inside the fma: one rounding of it less
}

// Sums of vectors [v0, v1) of a row (kThreads threads; the whole CTA calls).  The
// listed tokens are taken out of the vectors first, so that a batch's arithmetic
// is straight code with one test for a new reference (with a branch on the mask
// in each vector's, 512 rows of 126464 tokens took 40 us, not 38; the slice's
// first 16 to 128 KB asked into L2 before the list is read changed nothing); a thread adds those
// that it looks after at the end.
template <int DT>
__device__ Share stream_sums(const char* row, int64_t V, int v0, int v1, float c, float c_lo, const uint32_t* bits,
                            const Mine& mine) {
    constexpr int EPV = Row<DT>::EPV;
    Share a = no_share();
    float top = -INFINITY, ref = -FLT_MAX;
    f2 rest = pack2(0.f, 0.f);
    const f2 c2 = pack2(c, c), lo2 = pack2(c_lo, c_lo);
    const int whole = (int)min((int64_t)v1, V / EPV);
    auto add = [&](auto& w, const int (&v)[sizeof(w) / 16]) {
        constexpr int N = sizeof(w) / 16;
        uint32_t in[N];
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int at = (v[u] - v0) * EPV;  // first token of the vector, from the slice's start
            in[u] = (bits[at >> 5] >> (at & 31)) & ((1u << EPV) - 1u);
        }
        float m = -INFINITY;
#pragma unroll
        for (int u = 0; u < N; ++u) {
            if (in[u]) w[u] = without<DT>(w[u], in[u]);
            m = max_nan(m, Row<DT>::vmax(w[u]));
        }
        top = max_nan(top, m);
        if ((m - ref) * c > kRebase) {
            const float e = ex2((ref - m) * c);
            rest = mul2(rest, pack2(e, e));
            ref = m;
        }
        const f2 r2 = pack2(ref, ref);
        f2 sum[N];
#pragma unroll
        for (int u = 0; u < N; ++u) {
            float z[EPV];
            Row<DT>::unpack(w[u], z);
            f2 e[EPV / 2];
#pragma unroll
            for (int p = 0; p < EPV / 2; ++p) e[p] = weights_of(pack2(z[2 * p], z[2 * p + 1]), r2, c2, lo2);
#pragma unroll
            for (int h = EPV / 4; h; h >>= 1)
#pragma unroll
                for (int p = 0; p < h; ++p) e[p] = add2(e[p], e[p + h]);
            sum[u] = e[0];
        }
#pragma unroll
        for (int h = N / 2; h; h >>= 1)
#pragma unroll
            for (int u = 0; u < h; ++u) sum[u] = add2(sum[u], sum[u + h]);
        rest = add2(rest, sum[0]);
    };
    int v = v0 + (int)threadIdx.x;
    const uint4* vec = reinterpret_cast<const uint4*>(row);
    for (; v + (kUnroll - 1) * kThreads < whole; v += kUnroll * kThreads) {
        uint4 w[kUnroll];
        int at[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) at[u] = v + u * kThreads, w[u] = ld_row(vec + at[u]);
        add(w, at);
    }
    for (; v < v1; v += kThreads) {
        uint4 w[1] = {v < whole ? ld_row(vec + v) : load_vec<DT>(row, V, v)};
        const int at[1] = {v};
        add(w, at);
    }
    a.rest_ref = top;
    a.rest = rebased(hsum2(rest), ref, top, c);
    int at = kMine;
#pragma unroll
    for (int i = 0; i < kMine; ++i)
        if ((mine.own >> i) & 1u) {
            if (mine.s[i] > a.ref) at = i;
            a.ref = max_nan(a.ref, mine.s[i]);
        }
#pragma unroll
    for (int i = 0; i < kMine; ++i)
        if (((mine.own >> i) & 1u) && i != at) a.listed += ex2((mine.s[i] - or_zero(a.ref)) * c);
    return a;
}

// The row's sums over all the CTAs of its cluster, in every thread.  Each warp leaves
// its share in every CTA (a remote store needs no answer), one barrier later each
// warp adds up all of them for itself, and nothing remote is read, so no CTA has to
// outlive another.  started() comes before: no share is sent to a CTA that does not
// run yet.
__device__ __forceinline__ Total merge_row(const Cluster& cl, Shared& sh, Share a, float c, bool& twice) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    a = warp_share(a, c);
    if (cl.split > 1) {
        if (lane < cl.split) *cl.at(&sh.part[cl.rank * kWarps + warp], lane) = a;
        cl.sync();
    } else {
        if (lane == 0) sh.part[warp] = a;
        __syncthreads();
    }
    const int n = cl.split * kWarps;
    a = lane < n ? sh.part[lane] : no_share();
    for (int i = lane + 32; i < n; i += 32) {
        const Share b = sh.part[i];
        const float ref = max_nan(a.ref, b.ref), rest_ref = max_nan(a.rest_ref, b.rest_ref);
        const float a1 = b.ref > a.ref ? 1.f : 0.f, b1 = 1.f - a1;  // whose 1 counts now
        const float listed = rebased(fabsf(a.listed) + a1, a.ref, ref, c) + rebased(fabsf(b.listed) + b1, b.ref, ref, c);
        a.listed = is_twice(a.listed) || is_twice(b.listed) ? -listed : listed;
        a.rest = rebased(a.rest, a.rest_ref, rest_ref, c) + rebased(b.rest, b.rest_ref, rest_ref, c);
        a.ref = ref;
        a.rest_ref = rest_ref;
    }
    a = warp_share(a, c);
    Total q;
    q.mx = max_nan(a.ref, a.rest_ref);
    q.rest_ref = a.rest_ref;
    q.rest = a.rest;
    q.up = ex2((a.rest_ref - or_zero(q.mx)) * c);
    const float listed = fabsf(a.listed), rest = q.rest * q.up;
    q.all = rebased(1.f + listed, a.ref, q.mx, c) + rest;
    q.away = a.ref == q.mx ? (listed + rest) / q.all : -1.f;
    twice = is_twice(a.listed);
    return q;
}
// The cluster's CTAs run: every thread says so first and, before it stores into
// another CTA, waits for the others.
__device__ __forceinline__ void started(const Cluster& cl) {
    if (cl.split > 1) cg::this_cluster().barrier_arrive();
}
__device__ __forceinline__ void all_started(const Cluster& cl) {
    if (cl.split > 1) cg::this_cluster().barrier_wait();
}

// One float to storage.
template <int DT>
__device__ __forceinline__ void store_elem(void* row, int64_t i, float x) {
    if constexpr (DT == DLM_F32)
        static_cast<float*>(row)[i] = x;
    else if constexpr (DT == DLM_BF16)
        static_cast<__nv_bfloat16*>(row)[i] = __float2bfloat16_rn(x);
    else
        static_cast<__half*>(row)[i] = __float2half_rn(x);
}

// scale * 2^((z - m) c) of a vector, in storage.
struct Slope {
    f2 m, c, scale;
    __device__ Slope(float m1, float c1, float s1) : m(pack2(m1, m1)), c(pack2(c1, c1)), scale(pack2(s1, s1)) {}
};
template <int DT>
__device__ __forceinline__ uint4 slope_of(uint4 w, const Slope& s) {
    constexpr int EPV = Row<DT>::EPV;
    float z[EPV];
    Row<DT>::unpack(w, z);
    uint32_t r[4];
#pragma unroll
    for (int p = 0; p < EPV / 2; ++p) {
        float x, y;
        unpack2(mul2(ex2x2(mul2(sub2(pack2(z[2 * p], z[2 * p + 1]), s.m), s.c)), s.scale), x, y);
        if constexpr (DT == DLM_F32) {
            r[2 * p] = __float_as_uint(x);
            r[2 * p + 1] = __float_as_uint(y);
        } else if constexpr (DT == DLM_BF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
            r[p] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __half2 h = __floats2half2_rn(x, y);
            r[p] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// scale * 2^((z - m) c) for vectors [v0, v1) of the row; scale = 0 writes
// zeros without reading.  In place is fine: a vector is read before it is
// written, by the same thread.
template <int DT>
__device__ void stream_grad(const char* row, char* out, int64_t V, int v0, int v1, float m, float c, float scale) {
    constexpr int EPV = Row<DT>::EPV;
    const int whole = (int)min((int64_t)v1, V / EPV);
    const Slope slope(m, c, scale);
    auto value = [&](uint4 w) { return slope_of<DT>(w, slope); };
    const uint4* src = reinterpret_cast<const uint4*>(row);
    uint4* dst = reinterpret_cast<uint4*>(out);
    int v = v0 + (int)threadIdx.x;
    if (scale == 0.f) {
        for (; v < whole; v += kThreads) st_row(dst + v, make_uint4(0, 0, 0, 0));
    } else {
        for (; v + (kUnroll - 1) * kThreads < whole; v += kUnroll * kThreads) {
            uint4 w[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) w[u] = ld_row(src + v + u * kThreads);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) st_row(dst + v + u * kThreads, value(w[u]));
        }
        for (; v < whole; v += kThreads) st_row(dst + v, value(ld_row(src + v)));
    }
    if (v1 > whole) {  // the row's last, cut vector
        for (int64_t i = (int64_t)whole * EPV + threadIdx.x; i < V; i += kThreads)
            store_elem<DT>(out, i, scale == 0.f ? 0.f : scale * ex2((Row<DT>::scalar(row, i) - m) * c));
    }
}

// What the listed tokens' gradient needs of the row.
struct Listed {
    float m, inv, inv_p, away, lse_t;
    bool twice, rest;
};

// 1 - p_v of the token that entry j lists, to all digits however near p_v is to 1:
// without the rest the other entries' sum, with it the series of 1 - e^-d.  (A token
// that is listed in parts, with the rest: one less the integer weights, to 2^-45.)
__device__ __forceinline__ float teacher_away(const DistillArgs& a, const List& l, const Shared& sh, int j, const Listed& row) {
    const int id = l.id[j], K = a.k;
    if (!row.rest) {
        float others = 0.f;
#pragma unroll 8
        for (int i = 0; i < K; ++i) others += l.id[i] != id ? l.p[i] : 0.f;
        return others * row.inv_p;
    }
    const WeightScale ws = teacher_scale(a, sh);
    float y, lo;
    if (!row.twice) {
        const double d = (double)row.lse_t - (double)l.t[j] * a.inv_t;
        if (fabs(d) < 0x1p-12) return (float)one_less_exp(d);
    }
    uint64_t w = 0;
    for (int i = row.twice ? 0 : j; i < (row.twice ? K : j + 1); ++i)
        if (l.id[i] == id) w += teacher_weight(a, l.t[i], ws, true, row.lse_t, y, lo);
    return (float)(int64_t)((1ull << kWeightBits) - w) * kUnit;
}

// The listed tokens of this CTA's slice [e0, e1): g (q_v - p_v), for a token that
// the student is sure of g ((1 - p_v) - (1 - q_v)).  An id that is listed more than
// once (`twice`: maybe) is written by its first entry, with the sum of all of them.
template <int DT>
__device__ __forceinline__ void write_listed(const DistillArgs& a, const List& l, const Shared& sh, char* out, int e0,
                                             int e1, const Listed& row, float g) {
    const int K = a.k;
    for (int j = threadIdx.x; j < K; j += kThreads) {
        const int id = l.id[j];
        if (id < e0 || id >= e1) continue;
        float p = l.p[j], s = l.s[j];
        bool first = true;
        if (row.twice) {
            p = 0.f;
            for (int i = 0; i < K; ++i) {
                if (l.id[i] != id) continue;
                first &= i >= j;
                p += l.p[i];
                s = max_nan(s, l.s[i]);  // (one of them has the logit, the others it or -inf)
            }
        }
        if (!first) continue;
        const float q = row.inv * ex2((s - row.m) * a.scale);
        float slope = q - p * row.inv_p;
        if (q > 0.5f && s == row.m) slope = teacher_away(a, l, sh, j, row) - row.away;
        store_elem<DT>(out, id, g * slope);
    }
}

template <int DT>
struct Slice {
    int v0, v1;       // vectors of this CTA
    int e0, e1;       // its tokens
    __device__ Slice(int64_t V, const Cluster& cl) {
        constexpr int EPV = Row<DT>::EPV;
        const int nv = (int)((V + EPV - 1) / EPV);
        // whole words of the bitmap per slice: 32 / EPV vectors each
        const int unit = 32 / EPV;
        const int per = ((nv + cl.split - 1) / cl.split + unit - 1) / unit * unit;
        v0 = min(nv, cl.rank * per);
        v1 = min(nv, v0 + per);
        e0 = v0 * EPV;
        e1 = min((int)V, v1 * EPV);
    }
};

// The loss of a row, and with GRAD (rows too long for distill_row_kernel) the
// gradient of the sum of the row losses.
template <int DT, bool REST, bool GRAD>
__global__ void __launch_bounds__(kThreads, 4) distill_stream_kernel(const DistillArgs a) {
    extern __shared__ __align__(16) unsigned char s_raw[];
    Shared& sh = *reinterpret_cast<Shared*>(s_raw);
    const List l = carve(s_raw, a.k);
    const int t = threadIdx.x, K = a.k;
    Cluster cl;
    cl.split = a.split;
    const int64_t r = blockIdx.x / a.split;
    cl.rank = (int)(blockIdx.x - r * a.split);
    const int64_t V = a.vocab;
    const char* row = static_cast<const char*>(a.student) + r * a.row_stride * Row<DT>::ESZ;
    char* out = GRAD ? static_cast<char*>(a.grad) + r * a.grad_stride * Row<DT>::ESZ : nullptr;
    const Slice<DT> sl(V, cl);
    const int id0 = t < K ? a.ids[r * K + t] : -1;
    const float x0 = t < K ? teacher_at(a, r * K + t) : 0.f;
    const float weight = a.weights ? a.weights[r] : 1.f;
    const float lse_t = REST ? a.teacher_lse[r] : 0.f;
    const float c = a.scale;
    if (weight == 0.f) {  // the row has no loss: it is not read
        if (cl.rank == 0 && t == 0) {
            a.loss[r] = 0.f;
            write_state(a.state ? a.state + r * DLM_DISTILL_STATE : nullptr, Total{}, 0.f, 0.f, 0.f, 0.f, false);
        }
        if (GRAD) stream_grad<DT>(row, out, V, sl.v0, sl.v1, 0.f, c, 0.f);
        return;
    }
    started(cl);
    for (int i = t; i < (int)((sl.e1 - sl.e0 + 31) / 32); i += kThreads) l.bits[i] = 0;
    list_load(a, l, sh, r, lse_t, id0, x0);
    __syncthreads();
    Mine mine;
    mark_listed(l, K, sl.e0, sl.e1, mine);
    // the listed logits are asked for now and used after the stream
#pragma unroll
    for (int i = 0; i < kMine; ++i)
        mine.s[i] = (mine.in >> i) & 1u ? Row<DT>::scalar(row, l.id[t + i * kThreads]) : 0.f;
    list_weigh(a, l, sh, REST, lse_t);
    if (__syncthreads_or(mine.in != mine.own)) lowest_own(l, K, mine);
    Share share = stream_sums<DT>(row, V, sl.v0, sl.v1, c, a.scale_lo, l.bits, mine);
    if (mine.in != mine.own) share.listed = -share.listed;
    all_started(cl);
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        if (!((mine.in >> i) & 1u)) continue;
        const int j = t + i * kThreads;
        l.s[j] = mine.s[i];
        if (cl.rank != 0) cl.at(l.s, 0)[j] = mine.s[i];
    }
    bool twice;
    const Total all = merge_row(cl, sh, share, c, twice);
    const Teacher tch = list_total(sh, REST);
    float inv, base, tail;
    row_factors(tch, all, REST, inv, base, tail);
    if (cl.rank == 0) {
        if (t == 0)
            write_state(a.state ? a.state + r * DLM_DISTILL_STATE : nullptr, all, inv, base, tail, lse_t, REST);
        finish_loss(a, l, sh, tch, r, weight, all, REST, lse_t, twice);
    }
    if (GRAD) {
        const float g = weight * (float)a.inv_t;
        stream_grad<DT>(row, out, V, sl.v0, sl.v1, base, c, g * tail);
        __syncthreads();
        if (inv != 0.f)
            write_listed<DT>(a, l, sh, out, sl.e0, sl.e1, Listed{all.mx, inv, tch.inv, all.away, lse_t, true, REST}, g);
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads) distill_stream_grad_kernel(const DistillArgs a) {
    extern __shared__ __align__(16) unsigned char s_raw[];
    Shared& sh = *reinterpret_cast<Shared*>(s_raw);
    const List l = carve(s_raw, a.k);
    const int t = threadIdx.x, K = a.k;
    Cluster cl;
    cl.split = a.split;
    const int64_t r = blockIdx.x / a.split;
    cl.rank = (int)(blockIdx.x - r * a.split);
    const int64_t V = a.vocab;
    const char* row = static_cast<const char*>(a.student) + r * a.row_stride * Row<DT>::ESZ;
    char* out = static_cast<char*>(a.grad) + r * a.grad_stride * Row<DT>::ESZ;
    const Slice<DT> sl(V, cl);
    const float g = (a.weights ? a.weights[r] : 1.f) * (a.grad_loss ? a.grad_loss[r] : 1.f) * (float)a.inv_t;
    const float c = a.scale;
    const float* state = a.state + r * DLM_DISTILL_STATE;
    const float m = state[0], inv = state[1], tail = state[2], base = state[5];
    const bool rest = state[4] != 0.f;
    if (g == 0.f || inv == 0.f) {
        stream_grad<DT>(row, out, V, sl.v0, sl.v1, m, c, 0.f);
        return;
    }
    list_load(a, l, sh, r, state[3], t < K ? a.ids[r * K + t] : -1, t < K ? teacher_at(a, r * K + t) : 0.f);
    __syncthreads();
    list_weigh(a, l, sh, rest, state[3]);
    for (int j = t; j < K; j += kThreads) {
        const int id = l.id[j];
        if (id >= sl.e0 && id < sl.e1) l.s[j] = Row<DT>::scalar(row, id);
    }
    __syncthreads();
    const Teacher tch = list_total(sh, rest);
    stream_grad<DT>(row, out, V, sl.v0, sl.v1, base, c, g * tail);
    __syncthreads();
    write_listed<DT>(a, l, sh, out, sl.e0, sl.e1, Listed{m, inv, tch.inv, state[6], state[3], true, rest}, g);
}

// ---- the row on chip --------------------------------------------------------

// Takes element e out of a slice in shared memory: its value, and -inf in its
// place.  -inf if that was there already (an id listed twice, or a logit that
// carries nothing).
template <int DT>
__device__ __forceinline__ float take_out(uint4* data, int e) {
    if constexpr (DT == DLM_F32) {
        return __uint_as_float(atomicExch(reinterpret_cast<uint32_t*>(data) + e, 0xff800000u));
    } else {
        uint32_t* w = reinterpret_cast<uint32_t*>(data) + (e >> 1);
        const int shift = (e & 1) * 16;
        const uint32_t half = 0xffffu << shift, gone = Row<DT>::kNegInf << shift;
        uint32_t old = *w, seen;
        do {
            seen = old;
            old = atomicCAS(w, seen, (seen & ~half) | gone);
        } while (old != seen);
        const uint16_t bits = (uint16_t)(seen >> shift);
        return Row<DT>::scalar(&bits, 0);
    }
}

// Where a token of the slice is listed again, its lowest entry gets the logit that one
// of them took by chance (as in lowest_own).  Returns the thread's largest.
__device__ __forceinline__ float settle_own(const List& l, int K, int e0, int e1) {
    for (int j = threadIdx.x; j < K; j += kThreads) {
        const int id = l.id[j];
        if (id < e0 || id >= e1 || !l.own[j]) continue;
        int at = 0;
        while (l.id[at] != id) ++at;
        if (at == j) continue;
        l.s[at] = l.s[j];
        l.own[at] = 1;
        l.own[j] = 0;
    }
    __syncthreads();
    float top = -INFINITY;
    for (int j = threadIdx.x; j < K; j += kThreads)
        if (l.id[j] >= e0 && l.id[j] < e1 && l.own[j]) top = max_nan(top, l.s[j]);
    return top;
}

// SUMS: loss and the gradient of the losses' sum; else the gradient from the
// state (REST says nothing there).
template <int DT, bool REST, bool SUMS>
__global__ void __launch_bounds__(kThreads, 5) distill_row_kernel(const DistillArgs a) {
    extern __shared__ __align__(16) unsigned char s_raw[];
    constexpr int EPV = Row<DT>::EPV;
    Shared& sh = *reinterpret_cast<Shared*>(s_raw);
    const List l = carve(s_raw, a.k);
    const int t = threadIdx.x, K = a.k;
    Cluster cl;
    cl.split = a.split;
    const int64_t r = blockIdx.x / a.split;
    cl.rank = (int)(blockIdx.x - r * a.split);
    const int64_t V = a.vocab;
    const char* row = static_cast<const char*>(a.student) + r * a.row_stride * Row<DT>::ESZ;
    char* out = static_cast<char*>(a.grad) + r * a.grad_stride * Row<DT>::ESZ;
    const Slice<DT> sl(V, cl);
    const int n = sl.v1 - sl.v0, whole = (int)min((int64_t)sl.v1, V / EPV) - sl.v0;  // vectors; those not cut by V
    uint4* data = reinterpret_cast<uint4*>(s_raw + slice_offset(K));
    const float c = a.scale;
    const int id0 = t < K ? a.ids[r * K + t] : -1;
    const float x0 = t < K ? teacher_at(a, r * K + t) : 0.f;
    const float weight = a.weights ? a.weights[r] : 1.f;
    float g = weight * (float)a.inv_t, m = 0.f, inv = 0.f, base = 0.f, tail = 0.f, lse_t = 0.f;
    bool rest = REST;
    if (SUMS) {
        if (REST) lse_t = a.teacher_lse[r];
    } else {
        const float* state = a.state + r * DLM_DISTILL_STATE;
        m = state[0];
        inv = state[1];
        tail = state[2];
        lse_t = state[3];
        rest = state[4] != 0.f;
        base = state[5];
        if (a.grad_loss) g *= a.grad_loss[r];
    }
    if (SUMS ? weight == 0.f : (g == 0.f || inv == 0.f)) {  // no gradient: the row is not read
        if (SUMS && cl.rank == 0 && t == 0) a.loss[r] = 0.f;
        stream_grad<DT>(row, out, V, sl.v0, sl.v1, 0.f, c, 0.f);
        return;
    }
    if (SUMS) started(cl);
    // the slice: every thread copies, and later reads, its own vectors
    const uint4* src = reinterpret_cast<const uint4*>(row) + sl.v0;
    for (int v = t; v < whole; v += kThreads) cp_async16(data + v, src + v);
    if (whole < n && t == 0) data[whole] = load_vec<DT>(row, V, sl.v0 + whole);  // the row's last, cut vector
    list_load(a, l, sh, r, lse_t, id0, x0);
    __syncthreads();
    list_weigh(a, l, sh, rest, lse_t);
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    // the listed tokens leave the slice; one entry of each has its logit
    bool twice = false;
    float top = -INFINITY;
    for (int j = t; j < K; j += kThreads) {
        const int id = l.id[j];
        if (id < sl.e0 || id >= sl.e1) continue;
        const float s = take_out<DT>(data, (int)(id - sl.e0));
        const bool took = !(s == -INFINITY);
        l.s[j] = s;
        l.own[j] = took;
        twice |= !took;
        if (took) top = max_nan(top, s);
    }
    if (SUMS) {
        if (__syncthreads_or(twice)) top = settle_own(l, K, sl.e0, sl.e1);
        float high = -INFINITY;
        for (int v = t; v < n; v += kThreads) high = max_nan(high, Row<DT>::vmax(data[v]));
        const float ref = or_zero(high);  // nothing but -inf: weights of 0
        const f2 r2 = pack2(ref, ref), c2 = pack2(c, c), lo2 = pack2(a.scale_lo, a.scale_lo);
        f2 others = pack2(0.f, 0.f);
        for (int v = t; v < n; v += kThreads) {
            float z[EPV];
            Row<DT>::unpack(data[v], z);
            f2 e[EPV / 2];
#pragma unroll
            for (int p = 0; p < EPV / 2; ++p) e[p] = weights_of(pack2(z[2 * p], z[2 * p + 1]), r2, c2, lo2);
#pragma unroll
            for (int h = EPV / 4; h; h >>= 1)
#pragma unroll
                for (int p = 0; p < h; ++p) e[p] = add2(e[p], e[p + h]);
            others = add2(others, e[0]);
        }
        const float rest_sum = hsum2(others);
        // the listed tokens' weights; their logits to the first CTA
        float own = 0.f;
        bool first = true;
        all_started(cl);
        for (int j = t; j < K; j += kThreads) {
            const int id = l.id[j];
            if (id < sl.e0 || id >= sl.e1) continue;
            float s = l.s[j];
            if (l.own[j]) {
                if (s == top && first)
                    first = false;
                else
                    own += ex2((s - or_zero(top)) * c);
            } else {  // another entry has this token's logit, or it is -inf
                for (int i = 0; i < K; ++i)
                    if (l.id[i] == id && l.own[i]) s = l.s[i];
            }
            if (cl.rank != 0 || !l.own[j]) cl.at(l.s, 0)[j] = s;
        }
        const Total all = merge_row(cl, sh, Share{top, twice ? -own : own, high, rest_sum}, c, twice);
        row_factors(list_total(sh, REST), all, REST, inv, base, tail);
        m = all.mx;
        if (t == 0) {
            sh.row = all;
            sh.weight = weight;
            sh.lse_t = lse_t;
        }
    } else {
        if (t == 0) {
            sh.row.away = a.state[r * DLM_DISTILL_STATE + 6];
            sh.lse_t = lse_t;
        }
        twice = __syncthreads_or(twice);
    }
    const Teacher tch = list_total(sh, rest);
    const float scale = g * tail;
    uint4* dst = reinterpret_cast<uint4*>(out) + sl.v0;
    const Slope slope(base, c, scale);
#pragma unroll 2
    for (int v = t; v < whole; v += kThreads) st_row(dst + v, slope_of<DT>(data[v], slope));
    if (whole < n) {  // the row's last, cut vector
        for (int64_t i = (int64_t)(sl.v0 + whole) * EPV + t; i < V; i += kThreads)
            store_elem<DT>(out, i, scale * ex2((Row<DT>::scalar(data, i - sl.e0) - base) * c));
    }
    __syncthreads();
    if (inv != 0.f) write_listed<DT>(a, l, sh, out, sl.e0, sl.e1, Listed{m, inv, tch.inv, sh.row.away, sh.lse_t, twice, rest}, g);
    // (last: the gradient does not wait for it)
    if (SUMS && cl.rank == 0) finish_loss(a, l, sh, list_total(sh, REST), r, sh.weight, sh.row, REST, sh.lse_t, twice);
}

// Shared memory of a CTA that streams: the list, and with `bits` the bitmap of
// its slice.
size_t stream_bytes(int64_t V, int k, int split, bool bits) {
    size_t n = shared_bytes() + (size_t)k * 16;
    if (bits) n += (size_t)((V + split - 1) / split + 64) / 32 * 4 + 16;
    return n;
}

// The largest slice that a CTA can hold, and the one it should: five CTAs per SM.
constexpr int kMaxSlice = 190 * 1024, kGoodSlice = 39 * 1024;
constexpr int kMostShared = 227 * 1024;

template <typename F>
cudaError_t launch_rows(F kernel, const DistillArgs& a, size_t smem, cudaStream_t st) {
    if (smem > 48 * 1024) {  // the same limit whatever the call's size: calls may run side by side
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.n_rows * a.split));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.split > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int DT, bool REST>
cudaError_t launch_loss(const DistillArgs& a, cudaStream_t st) {
    const size_t smem = stream_bytes(a.vocab, a.k, a.split, true);
    if (!a.grad) return launch_rows(distill_stream_kernel<DT, REST, false>, a, smem, st);
    if (a.slice_vecs == 0) return launch_rows(distill_stream_kernel<DT, REST, true>, a, smem, st);
    return launch_rows(distill_row_kernel<DT, REST, true>, a, slice_offset(a.k) + (size_t)a.slice_vecs * 16, st);
}

template <int DT>
cudaError_t launch_grad(const DistillArgs& a, cudaStream_t st) {
    if (a.slice_vecs == 0)
        return launch_rows(distill_stream_grad_kernel<DT>, a, stream_bytes(a.vocab, a.k, a.split, false), st);
    return launch_rows(distill_row_kernel<DT, false, false>, a, slice_offset(a.k) + (size_t)a.slice_vecs * 16, st);
}

}  // namespace

// CTAs per row, and for the gradient vectors per slice (0: the row is streamed).
// A slice of about 40 KB lets five CTAs share an SM; rows too few to fill the
// GPU are cut finer, down to 8 KB.  The loss alone splits a row only when the
// rows do not fill the GPU and each thread still gets two batches of vectors.
void distill_plan(DistillArgs& a, int dtype, int num_sms) {
    const int epv = dtype == DLM_F32 ? 4 : 8, unit = 32 / epv;
    const int64_t nv = (a.vocab + epv - 1) / epv;
    int split = 1;
    a.slice_vecs = 0;
    if (a.grad) {
        auto slice = [&](int n) { return ((nv + n - 1) / n + unit - 1) / unit * unit; };
        while (split < 8 && slice(split) * 16 > kGoodSlice) split *= 2;
        while (split < 8 && a.n_rows * split < 2LL * num_sms && slice(split) * 16 > 8 * 1024) split *= 2;
        if (slice(split) * 16 <= kMaxSlice) a.slice_vecs = (int)slice(split);
    } else {
        while (split < 8 && a.n_rows * split < 2LL * num_sms && nv / (split * 2) >= 2LL * kThreads) split *= 2;
    }
    a.split = split;
}

cudaError_t launch_distill_loss(const DistillArgs& a, int dtype, cudaStream_t st) {
    const bool rest = a.teacher_lse != nullptr;
    switch (dtype) {
    case DLM_BF16: return rest ? launch_loss<DLM_BF16, true>(a, st) : launch_loss<DLM_BF16, false>(a, st);
    case DLM_F16: return rest ? launch_loss<DLM_F16, true>(a, st) : launch_loss<DLM_F16, false>(a, st);
    default: return rest ? launch_loss<DLM_F32, true>(a, st) : launch_loss<DLM_F32, false>(a, st);
    }
}

cudaError_t launch_distill_grad(const DistillArgs& a, int dtype, cudaStream_t st) {
    switch (dtype) {
    case DLM_BF16: return launch_grad<DLM_BF16>(a, st);
    case DLM_F16: return launch_grad<DLM_F16>(a, st);
    default: return launch_grad<DLM_F32>(a, st);
    }
}

}  // namespace dlm
