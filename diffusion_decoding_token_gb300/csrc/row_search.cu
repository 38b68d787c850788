// row_search.cu -- the largest logits of a row, and a token sampled from it.
//
// row_topk: the first k of the order (logit descending, position ascending)
// and the row's log-sum-exp.  row_sample: temperature, top-k, top-p, min-p and
// one uniform number per row; every filter keeps a prefix of that same order,
// so a row's filters come down to one cut in it, and the token is the first
// position, in vocabulary order, whose running sum of kept weights exceeds u
// times their total.
//
// Both are bound by reading the row once from HBM, so the first pass over it
// leaves just enough behind to avoid reading it again: per run of 32 vectors
// (512 bytes) the maximum, and per batch of four runs the sum of the softmax
// weights relative to the batch's own maximum.  The k-th largest run maximum
// c is at most the k-th largest logit, so all of the top k lie in runs whose
// maximum is >= c: only those few runs are read again (from L2).  The
// candidates are decided with 64-bit integer weights (weight.cuh).
//
// Tokens that no short list can decide (a nucleus of thousands of tokens on a
// flat row, or no filter at all) are decided from sums over the row, in tiers.
// A tier knows how far its sums may be off; a token whose borders lie further
// than that from the target is the answer, otherwise the next tier looks:
//   0  the first pass's batch sums (off by 2^-18; no filter only);
//   1  one more pass with the exponent split into integer and fraction (2^-20.8);
//   2  the same with the fraction's power from a table of exact values, summed
//      as integers, and a small correction in 32 bits (2^-27);
//   3  the same with integer weights (2^-36).
// The passes of tiers 1 to 3 find the nucleus' end by a bracket: a sample of
// the row says between which two logits it must lie, the pass sums what is
// above, lists what is inside, and the list is sorted.  What the bracket
// misses (ties by the thousand, a top-k beyond the list) goes to a search by
// radix passes over the ordered keys, with counts (top-k) or integer masses.
//
// A row is worked by one CTA, or by a cluster of CTAs when rows are few.  With
// one CTA per row the rows that need another pass are left to a second launch
// that works each with a cluster: alone, a CTA would be at such a row long after
// all the others have ended.
//
// Measured (empty L2, 2048 bf16 rows of 152064 unless said; the rows' bytes at the
// card's 6.8 TB/s take 92 us): the 64 largest 149 us, 4.2 TB/s (the pass over the
// rows alone 105 to 111; a list is made while its CTA reads nothing); settings of
// their own per row 263 us; top_p = 0.95 at temperature 1 over rows of 126464, two
// of five of them flat, 482 us; 32 of those rows at 0.7 and 0.9, 61 us, a chain of
// a dozen steps of 1 to 8 us each; 32 rows of 1024, 13 us.  Four CTAs per SM (64
// registers): three took 157 us for the first of these, five and six 165 and 236
// with spills.
#include "common.cuh"
#include "launch.h"
#include "row_vec.cuh"
#include "weight.cuh"

namespace dlm {

namespace {

constexpr int kThreads = kRowThreads;
constexpr int kWarps = kRowWarps;
constexpr int kRuns = 4;               // runs (of 32 vectors) per batch
constexpr int kBatchVecs = 32 * kRuns;
constexpr int kCap = 2048;             // candidates held in shared memory
constexpr int kBracketCap = 2 * kCap;  // tokens of a bracket (the weights' space too)
constexpr int kSortBins = 1024;        // bins of a sort
constexpr int kFine = 1024;            // bins that a bracket's tokens are sorted into
constexpr int kListRuns = 128;         // run maxima that open a nucleus' candidate list
constexpr int kBracketSide = 1200;     // tokens on either side of its middle
constexpr int kSampleTokens = 16384;   // the sample that places a bracket
constexpr int kOpenSplit = 4;          // CTAs per row that the first launch left open
constexpr int kTries = 4;              // brackets that a row gets
constexpr int kListTopk = 1700;        // largest top-k whose list a sample's threshold can be trusted with
constexpr uint64_t kOne = 1ull << kWeightBits;
constexpr int kBins = 2048;            // radix bins of a pass over the whole row
constexpr uint32_t kKeyNegInf = 0x007fffffu;  // ordered key of -inf
static_assert(kCap == 8 * kThreads, "the longest list that is sorted");
static_assert(kFine % kThreads == 0 && kFine >= kThreads, "whole bins per thread");
static_assert(kCap >= 2 * DLM_MAX_TOPK, "a candidate list holds the largest top-k and ties");

// Keys whose unsigned order is the order of the floats; -0 counts as +0.
__device__ __forceinline__ uint32_t key_of(float z) {
    const uint32_t b = __float_as_uint(z + 0.0f);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// weight44 as a call: where it is met once or rarely, fifty instructions inline
// cost more to fetch than to run (a row that takes the long way runs most of its
// code once, and waited for instructions more than for anything but barriers).
__device__ __noinline__ uint64_t weight_call(float z, const WeightScale ws) { return weight44(z, ws); }

// What is to be done for a row: nothing more, a pass of tier 1, 2 or 3, a list
// of everything above a threshold, a pass of tier 1 around min-p's cut, or the
// radix search.
enum Verdict : int { kRadix = 0, kDone = 1, kTier1 = 2, kTier2 = 3, kTier3 = 4, kList = 5, kMinP = 6 };

// What one row's CTA (the first of its cluster) and the others share.
struct Ctrl {
    WeightScale ws;
    float top_p, min_p, u;
    int top_k;            // 0: off
    int bad;              // a parameter of this row is out of range
    int verdict;          // what the cluster does next
    uint32_t count;       // candidates found (may exceed the list)
    uint32_t runs;        // runs to read again
    int n;                // tokens kept, or -1
    uint64_t least;       // min-p: the smallest weight that stays
    uint64_t total;       // the row's mass, within margin
    uint64_t margin;
    uint64_t whole;       // a slice's mass, and the part of it above the bracket
    uint64_t top;
    uint64_t t_lo, t_mid, t_hi;  // what the bracket's tokens have to add: least, likely, most
    uint64_t err;
    int by_min;           // min-p's cut ends the row, not the nucleus
    float z_lo, z_hi;     // the bracket: z_lo <= z < z_hi
    int bin_lo, bin_hi;   // the same in 1/32 of an exponent below the maximum
    int tries;
    // the search over the whole row
    uint32_t prefix;      // key bits found so far
    uint64_t above;       // count or mass of the keys above the prefix
    uint32_t cut_key;     // kept: keys above cut_key, and of the positions at it
    uint32_t cut_ties;    // the first cut_ties that are <= cut_last
    uint32_t cut_last;
    uint64_t mass;        // kept mass
    uint64_t left;        // target inside the chosen batch
    uint64_t sure;        // bracket: the last candidate that surely stays, the mass
    uint64_t sure_mass;   // up to it, and up to the last one that may stay
    uint64_t slack;
    int batch;
    uint32_t ties_before;
    int first_bin, last_bin;
    int token;            // found by walk_batch
    float z;
    uint64_t lo_side, hi_side;
    int hits[2][kWarps];
    uint32_t first[kWarps];
    float wmax[8 * kWarps];  // the first pass's maximum of each warp of the cluster,
    float wmin[8 * kWarps];  // and its smallest (finite) run maximum
    int bins[kThreads];
    float fscan[kWarps];
    uint64_t scan[kWarps];
};

// Shared memory of a CTA.  tab: the weights' table.  buf[kCap] holds candidates or radix bins; wbuf[kCap]
// their weights, and behind buf the rest of a bracket's tokens.  sub[4 nb] and
// bsum[nb], the first pass's run maxima and batch sums, and bties[nb] of the
// radix search are used when wbuf is not and share its space.  fine[kFine]: the
// bins of a bracket, then the few tokens around its end.  bmass[nb] is the
// batches' mass; while runs are read again the list of them lies there.
struct Smem {
    Ctrl* c;
    uint64_t* tab;
    uint64_t* buf;
    uint64_t* wbuf;
    uint64_t* fine;
    uint64_t* bmass;
    uint16_t* runs;
    uint32_t* bties;
    float* sub;
    float* bsum;
};

__host__ __device__ inline size_t ctrl_bytes() { return (sizeof(Ctrl) + 15) & ~(size_t)15; }
__host__ __device__ inline size_t shared_space(int nb) {
    const size_t first = sizeof(float) * (size_t)nb * (kRuns + 2), list = sizeof(uint64_t) * kCap;
    return ((first > list ? first : list) + 15) & ~(size_t)15;
}

__device__ __forceinline__ Smem carve(unsigned char* p, int nb) {
    Smem s;
    s.c = reinterpret_cast<Ctrl*>(p);
    p += ctrl_bytes();
    s.tab = reinterpret_cast<uint64_t*>(p);
    p += sizeof(uint64_t) * 256;
    s.buf = reinterpret_cast<uint64_t*>(p);
    p += sizeof(uint64_t) * kCap;
    s.wbuf = reinterpret_cast<uint64_t*>(p);
    s.sub = reinterpret_cast<float*>(p);  // 16-byte aligned: a batch's four maxima are stored at once
    s.bsum = s.sub + nb * kRuns;
    s.bties = reinterpret_cast<uint32_t*>(s.bsum + nb);
    p += shared_space(nb);
    s.bmass = reinterpret_cast<uint64_t*>(p);
    s.runs = reinterpret_cast<uint16_t*>(p);
    p += sizeof(uint64_t) * nb;
    s.fine = reinterpret_cast<uint64_t*>(p);
    return s;
}

// (`fine` only where a bracket is worked)
size_t smem_bytes(int nb, bool fine) {
    return ctrl_bytes() + sizeof(uint64_t) * (256 + kCap + (fine ? kFine : 0) + (size_t)nb) + shared_space(nb);
}

// 64-bit sum in shared memory by two native 32-bit atomics: the carry of the
// lower half goes into the upper one.
__device__ __forceinline__ void shared_add(uint64_t* p, uint64_t v) {
    uint32_t* half = reinterpret_cast<uint32_t*>(p);
    const uint32_t lo = (uint32_t)v, old = atomicAdd(half, lo);
    const uint32_t hi = (uint32_t)(v >> 32) + (old + lo < old ? 1u : 0u);
    if (hi) atomicAdd(half + 1, hi);
}

// buf[0, 256 E) ascending: a bitonic network with E elements per thread in
// registers.  Steps within a thread's elements need nothing, steps within a
// warp's 32 E elements go by shuffles, and only those that reach further (6 of
// 66 for 2048) through shared memory.  (With every step in shared memory 2048
// elements took 91000 cycles.)
template <int E>
__device__ void bitonic(uint64_t* buf) {
    const int lane = threadIdx.x & 31, base = threadIdx.x * E;
    constexpr int M = kThreads * E;
    uint64_t x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = buf[base + e];
    for (int k = 2; k <= M; k <<= 1) {
        if (k > 32 * E) {
            __syncthreads();  // (the loads, or the last round's, are done)
#pragma unroll
            for (int e = 0; e < E; ++e) buf[base + e] = x[e];
            __syncthreads();
            for (int j = k >> 1; j >= 32 * E; j >>= 1) {
#pragma unroll
                for (int q = 0; q < E / 2; ++q) {
                    const int i = threadIdx.x + q * kThreads, lo = 2 * i - (i & (j - 1)), hi = lo + j;
                    const uint64_t u = buf[lo], v = buf[hi];
                    const bool swap = (u > v) == ((lo & k) == 0);
                    buf[lo] = swap ? v : u;
                    buf[hi] = swap ? u : v;
                }
                __syncthreads();
            }
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = buf[base + e];
        }
        for (int j = min(k >> 1, 16 * E); j >= E; j >>= 1) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const uint64_t y = __shfl_xor_sync(DLM_FULL_MASK, x[e], j / E);
                const bool up = ((base + e) & k) == 0, low = (lane & (j / E)) == 0;
                x[e] = (up == low) == (x[e] < y) ? x[e] : y;
            }
        }
#pragma unroll
        for (int j = E / 2; j > 0; j >>= 1) {
            if (2 * j > k) continue;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (e & j) continue;
                const bool up = ((base + e) & k) == 0;
                const uint64_t u = x[e], v = x[e + j];
                const bool swap = (u > v) == up;
                x[e] = swap ? v : u;
                x[e + j] = swap ? u : v;
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) buf[base + e] = x[e];
    __syncthreads();
}

// Sort buf[0, n) ascending (n <= kCap, entries differ).  Short lists by rank
// (every thread counts the smaller ones, broadcast reads, two barriers), longer
// ones by bins: the upper words between the smallest and the largest in
// kSortBins equal steps, the bins' starts from a scan, and each entry's rank
// among its bin's.  Equal steps of a candidate's word are narrow near 0, which
// suits a list's tail and an outlier; where logits of both signs are listed the
// steps are equal in the logit (651 rows of 1611, k = 575: 30 us for 54; with all
// lists so, the 1000 largest of 61 rows of 100003 floats take 50 us, not 44).
// Where many share a bin (ties), or there is no room for bins, the network,
// padded to a power of two (62 us for those 1000 largest; top_k = 1500 of 512
// rows of 152064: 415 us, 370 with bins).  `space` holds kSortBins words that are
// free, or is null.  (4 KB of their own for the bins cost the kernels more, 517
// us for 482 at 2048 rows of 126464: four CTAs' shared memory leaves that much
// less cache.)
__device__ __noinline__ void sort_u64(uint64_t* buf, int n, void* space, Ctrl* c) {
    if (n <= kThreads) {
        const int i = threadIdx.x;
        const uint64_t v = i < n ? buf[i] : 0;
        int r = 0;
        if (i < n)
            for (int j = 0; j < n; ++j) r += buf[j] < v;
        __syncthreads();
        if (i < n) buf[r] = v;
        __syncthreads();
        return;
    }
    if (space) {
        constexpr int E = kCap / kThreads, PER = kSortBins / kThreads;
        const int t = threadIdx.x;
        uint32_t* bins = static_cast<uint32_t*>(space);
        uint64_t x[E];
        uint32_t lo = 0xffffffffu, hi = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int i = t + e * kThreads;
            x[e] = i < n ? buf[i] : ~0ull;
            if (i < n) lo = min(lo, (uint32_t)(x[e] >> 32)), hi = max(hi, (uint32_t)(x[e] >> 32));
        }
        lo = __reduce_min_sync(DLM_FULL_MASK, lo);
        hi = __reduce_max_sync(DLM_FULL_MASK, hi);
        if ((t & 31) == 0) c->hits[0][t >> 5] = (int)lo, c->hits[1][t >> 5] = (int)hi;
#pragma unroll
        for (int j = 0; j < PER; ++j) bins[t + j * kThreads] = 0;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) lo = min(lo, (uint32_t)c->hits[0][w]), hi = max(hi, (uint32_t)c->hits[1][w]);
        // (conversion, difference and product are monotone, so bins are in order)
        const bool both = (lo ^ hi) >> 31;
        auto place_of = [&](uint32_t word) { return both ? -key_value(~word) : (float)word; };
        const float from = place_of(lo), step = (kSortBins - 0.5f) / fmaxf(place_of(hi) - from, 1e-30f);
        uint32_t at[E], most = 0;  // bin, and place in it
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (t + e * kThreads >= n) continue;
            const uint32_t bin = min((uint32_t)kSortBins - 1, (uint32_t)((place_of((uint32_t)(x[e] >> 32)) - from) * step));
            const uint32_t place = atomicAdd(&bins[bin], 1u);
            at[e] = bin << 16 | place;
            most = max(most, place);
        }
        if (!__syncthreads_or(most >= 64)) {
            uint32_t v[PER], sum = 0;
#pragma unroll
            for (int j = 0; j < PER; ++j) sum += v[j] = bins[t * PER + j];
            uint64_t all;
            uint32_t run = (uint32_t)block_scan((uint64_t)sum, c->scan, all);
#pragma unroll
            for (int j = 0; j < PER; ++j) {  // start and length
                bins[t * PER + j] = run << 16 | v[j];
                run += v[j];
            }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (t + e * kThreads < n) buf[(bins[at[e] >> 16] >> 16) + (at[e] & 0xffffu)] = x[e];
            __syncthreads();
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (t + e * kThreads >= n) continue;
                const uint32_t bin = bins[at[e] >> 16], i0 = bin >> 16, i1 = i0 + (bin & 0xffffu);
                uint32_t r = i0;
                for (uint32_t i = i0; i < i1; ++i) r += buf[i] < x[e];
                at[e] = r;
            }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (t + e * kThreads < n) buf[at[e]] = x[e];
            __syncthreads();
            return;
        }
    }
    const int m = n <= 2 * kThreads ? 2 * kThreads : n <= 4 * kThreads ? 4 * kThreads : 8 * kThreads;
    for (int i = n + threadIdx.x; i < m; i += kThreads) buf[i] = ~0ull;
    __syncthreads();
    if (m == 2 * kThreads)
        bitonic<2>(buf);
    else if (m == 4 * kThreads)
        bitonic<4>(buf);
    else
        bitonic<8>(buf);
}

// A candidate: sorts by logit descending, then position ascending.
__device__ __forceinline__ uint64_t candidate(float z, uint32_t i) { return ((uint64_t)(~key_of(z)) << 32) | i; }
__device__ __forceinline__ float candidate_value(uint64_t c) { return key_value(~(uint32_t)(c >> 32)); }

// A threshold that at least k of the n floats of `values` reach and few more
// (-inf when fewer than k are finite): counts in kThreads bins between the
// smallest and the largest, one barrier, and every warp adds the bins up from
// the top for itself.  (A search by bisection took a barrier a step; under a
// streaming load each cost the CTA about 1000 cycles.)  c->bins is zero before.
__device__ float threshold_for(const float* values, int n, int k, float lo, float hi, Ctrl* c) {
    if (n < k) return -INFINITY;
    const int lane = threadIdx.x & 31;
    const float scale = hi > lo ? fminf((float)kThreads / (hi - lo), 1e30f) : 0.f;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const float x = values[i];
        if (x > -INFINITY) atomicAdd(&c->bins[min(kThreads - 1, max(0, (int)((x - lo) * scale)))], 1);
    }
    __syncthreads();
    constexpr int PER = kThreads / 32;
    int v[PER], mine = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) mine += v[j] = c->bins[kThreads - 1 - (lane * PER + j)];
    int run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(DLM_FULL_MASK, run, o);
        if (lane >= o) run += x;
    }
    const uint32_t who = __ballot_sync(DLM_FULL_MASK, run >= k);
    if (!who) return -INFINITY;
    int at = 0, seen = run - mine;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        if (seen < k) at = kThreads - 1 - (lane * PER + j);
        seen += v[j];
    }
    at = __shfl_sync(DLM_FULL_MASK, at, __ffs(who) - 1);
    // a little below the bin's edge, so that nothing of it is lost to rounding
    return lo + (scale > 0.f ? (float)at / scale : 0.f) - 1e-6f * (fabsf(lo) + fabsf(hi));
}

// Keeps of the n > kThreads candidates in buf the first k of the order and few
// more, where that makes the list short enough to need no sort: the threshold
// search over the candidates' values, then the rest is copied out and back.
// Returns how many are left.
__device__ int top_candidates(const Smem& s, int n, int k) {
    if (n <= kThreads || k > kThreads * 3 / 4) return n;
    const int t = threadIdx.x;
    Ctrl* c = s.c;
    float* values = reinterpret_cast<float*>(s.wbuf);
    uint64_t* out = s.wbuf + kCap / 2;
    float lo = INFINITY;
    for (int i = t; i < n; i += kThreads) {
        const float x = candidate_value(s.buf[i]);
        values[i] = x;
        lo = fminf(lo, x);
    }
    if (t == 0) c->runs = 0;
    c->bins[t] = 0;
    lo = -block_max_nan(-lo, c->fscan);  // (its barriers order the rest too)
    const float least = threshold_for(values, n, k, lo, c->ws.m, c);
    for (int i = t; i < n; i += kThreads)
        if (values[i] >= least) {
            const uint32_t at = atomicAdd(&c->runs, 1u);
            if (at < (uint32_t)kThreads) out[at] = s.buf[i];
        }
    __syncthreads();
    const int left = (int)c->runs;
    if (left > kThreads) return n;  // ties
    if (t < left) s.buf[t] = out[t];
    __syncthreads();
    return left;
}

// Push the elements z >= least of one loaded vector of each lane (positions
// from pos0 on) into the list dst of `cap` entries, its length in *count.
template <int DT>
__device__ __forceinline__ void push(uint4 w, uint32_t pos0, float least, uint64_t* dst, uint32_t cap,
                                     uint32_t* count) {
    constexpr int EPV = Row<DT>::EPV;
    const int lane = threadIdx.x & 31;
    float z[EPV];
    Row<DT>::unpack(w, z);
    uint32_t mine = 0;
#pragma unroll
    for (int e = 0; e < EPV; ++e) mine |= (uint32_t)(z[e] >= least && z[e] > -INFINITY) << e;
    if (!__any_sync(DLM_FULL_MASK, mine != 0)) return;
    const int n = __popc(mine);
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(DLM_FULL_MASK, inc, o);
        if (lane >= o) inc += x;
    }
    uint32_t base = 0;
    if (lane == 31) base = atomicAdd(count, (uint32_t)inc);
    base = __shfl_sync(DLM_FULL_MASK, base, 31) + (uint32_t)(inc - n);
    if (mine) {
#pragma unroll
        for (int e = 0; e < EPV; ++e)
            if ((mine >> e) & 1u) {
                if (base < cap) dst[base] = candidate(z[e], pos0 + (uint32_t)e);
                ++base;
            }
    }
}

// The elements z >= least of the whole row into buf (c->count of them, which
// may exceed kCap): the runs whose maximum reaches it are listed first, then
// each warp reads four of them at a time.
template <int DT>
__device__ void gather_runs(const char* row, int64_t V, int nsub, const Smem& s, float least) {
    constexpr int EPV = Row<DT>::EPV;
    constexpr int kAhead = 4;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Ctrl* c = s.c;
    if (threadIdx.x == 0) c->runs = c->count = 0;
    __syncthreads();
    for (int i0 = warp * 32; i0 < nsub; i0 += kThreads) {
        const int i = i0 + lane;
        const bool hit = i < nsub && s.sub[i] >= least;
        const uint32_t who = __ballot_sync(DLM_FULL_MASK, hit);
        if (!who) continue;
        uint32_t base = 0;
        if (lane == 0) base = atomicAdd(&c->runs, (uint32_t)__popc(who));
        base = __shfl_sync(DLM_FULL_MASK, base, 0);
        if (hit) s.runs[base + __popc(who & ((1u << lane) - 1u))] = (uint16_t)i;
    }
    __syncthreads();
    const int n = (int)c->runs;
    for (int i = warp; i < n; i += kWarps * kAhead) {
        uint4 w[kAhead];
        int v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int at = i + j * kWarps;
            v[j] = at < n ? (int)s.runs[at] * 32 + lane : -1;
            if (at < n) w[j] = load_vec<DT>(row, V, v[j]);
        }
        uint32_t mask = 0;  // elements that go into the list, a bit each
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (v[j] < 0) continue;
            float z[EPV];
            Row<DT>::unpack(w[j], z);
#pragma unroll
            for (int e = 0; e < EPV; ++e) mask |= (uint32_t)(z[e] >= least && z[e] > -INFINITY) << (j * EPV + e);
        }
        const int mine = __popc(mask);
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(DLM_FULL_MASK, inc, o);
            if (lane >= o) inc += x;
        }
        uint32_t at = 0;
        if (lane == 31) at = atomicAdd(&c->count, (uint32_t)inc);
        at = __shfl_sync(DLM_FULL_MASK, at, 31) + (uint32_t)(inc - mine);
        if (!mask) continue;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (!((mask >> (j * EPV)) & ((1u << EPV) - 1u))) continue;
            float z[EPV];
            Row<DT>::unpack(w[j], z);
#pragma unroll
            for (int e = 0; e < EPV; ++e)
                if ((mask >> (j * EPV + e)) & 1u) {
                    if (at < (uint32_t)kCap) s.buf[at] = candidate(z[e], (uint32_t)(v[j] * EPV + e));
                    ++at;
                }
        }
    }
    __syncthreads();
}

// The same over every run of batches [b0, b1), into a list that may be
// another CTA's of the cluster.
template <int DT>
__device__ __noinline__ void gather_slice(const char* row, int64_t V, int b0, int b1, float least, uint64_t* dst,
                                          uint32_t* count) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, end = b1 * kRuns;
    auto fetch = [&](int i) { return i < end ? load_vec<DT>(row, V, i * 32 + lane) : make_uint4(0, 0, 0, 0); };
    int i = b0 * kRuns + warp;
    uint4 w0 = fetch(i), w1 = fetch(i + kWarps), w2 = fetch(i + 2 * kWarps);
#pragma unroll 1
    for (; i < end; i += kWarps) {
        const uint4 w = w0;
        w0 = w1;
        w1 = w2;
        w2 = fetch(i + 3 * kWarps);
        push<DT>(w, (uint32_t)((i * 32 + lane) * Row<DT>::EPV), least, dst, kCap, count);
    }
}

// ---- the first pass --------------------------------------------------------

// Run maxima of batches [b0, b1), and with `sums` each batch's sum of
// 2^((z - ref) c), ref the batch's maximum (a batch of -inf only sums to 0).
// The next batch is loaded while one is summed, and the first while `begin` finds
// out the scale (0: no sums; negative: leave).  Returns the warp's maximum, and
// in `low` its smallest run maximum that is finite.
template <int DT, typename F>
__device__ __forceinline__ float scan_rows(const char* row, int64_t V, int b0, int b1, F begin, float* sub,
                                           float* bsum, float& low) {
    constexpr int EPV = Row<DT>::EPV;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto fetch = [&](int b, uint4 (&w)[kRuns]) {
        const int v0 = b * kBatchVecs + lane;
        if ((int64_t)(b + 1) * kBatchVecs * EPV <= V) {
#pragma unroll
            for (int i = 0; i < kRuns; ++i) w[i] = ld_stream(reinterpret_cast<const uint4*>(row) + v0 + i * 32);
        } else {
#pragma unroll
            for (int i = 0; i < kRuns; ++i) w[i] = load_vec<DT>(row, V, v0 + i * 32);
        }
    };
    float most = -INFINITY;
    uint4 next[kRuns];
    if (b0 + warp < b1) fetch(b0 + warp, next);
    const float c = begin();
    const bool sums = c > 0.f;
    if (c < 0.f) return 0.f;
    for (int b = b0 + warp; b < b1; b += kWarps) {
        uint4 w[kRuns];
#pragma unroll
        for (int i = 0; i < kRuns; ++i) w[i] = next[i];
        if (b + kWarps < b1) fetch(b + kWarps, next);
        float m[kRuns];
#pragma unroll
        for (int i = 0; i < kRuns; ++i) m[i] = warp_max_nan(Row<DT>::vmax(w[i]));
        if (lane == 0) *reinterpret_cast<float4*>(sub + b * kRuns) = make_float4(m[0], m[1], m[2], m[3]);
        const float ref = max_nan(max_nan(m[0], m[1]), max_nan(m[2], m[3]));
        most = max_nan(most, ref);
#pragma unroll
        for (int i = 0; i < kRuns; ++i) low = fminf(low, m[i] > -INFINITY ? m[i] : INFINITY);
        if (!sums) continue;
        const float r = ref > -INFINITY ? ref : 0.f;  // -inf - 0 stays -inf: weight 0
        const f2 r2 = pack2(r, r), c2 = pack2(c, c);
        f2 acc[kRuns];
#pragma unroll
        for (int i = 0; i < kRuns; ++i) {
            float z[EPV];
            Row<DT>::unpack(w[i], z);
            f2 e[EPV / 2];
#pragma unroll
            for (int p = 0; p < EPV / 2; ++p) e[p] = ex2x2(mul2(sub2(pack2(z[2 * p], z[2 * p + 1]), r2), c2));
#pragma unroll
            for (int h = EPV / 4; h; h >>= 1)
#pragma unroll
                for (int p = 0; p < h; ++p) e[p] = add2(e[p], e[p + h]);
            acc[i] = e[0];
        }
        float s = hsum2(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])));
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(DLM_FULL_MASK, s, o);
        if (lane == 0) bsum[b] = s;
    }
    return most;
}

// A batch's sum relative to the row's maximum, in units of 2^-44.
__device__ __forceinline__ uint64_t batch_mass(const float* sub, const float* bsum, int b, const WeightScale& ws) {
    const float ref = fmaxf(fmaxf(sub[4 * b], sub[4 * b + 1]), fmaxf(sub[4 * b + 2], sub[4 * b + 3]));
    const float s = bsum[b] * ex2((ref - ws.m) * ws.c_hi);
    return ref > -INFINITY ? (uint64_t)__float2ull_rn(s * 17592186044416.0f) : 0ull;
}

// ---- candidates ------------------------------------------------------------

// Writes the row's token (thread-wise: the one thread that found it).
__device__ __forceinline__ void write_token(const RowSearchArgs& a, const Ctrl* c, int64_t o,
                                            int token, float z, uint64_t mass) {
    float lo;
    const float y = weight_exponent(z, c->ws, lo);
    // 2^-(y + lo) over the kept mass
    const float w = exp2f(-y) * fmaf(lo, -kLn2, 1.0f);
    a.token[o] = token;
    a.prob[o] = y < INFINITY ? fminf(1.0f, w / ((float)mass * 0x1p-44f)) : 0.f;
    if (a.conf) a.conf[o] = expf(z - a.lse_in[o]);
}

// A list's contract with the filters.
struct ListRule {
    int k;            // top-k (the list's length when it is off)
    bool complete;    // every token that top-k and min-p could keep is listed, and
                      // the mass that top_p is a share of is the k largest's; else
                      // it is c->total +- c->margin
    bool all_least;   // every token with a weight >= c->least is listed
};

// The mass of 2^20 - 1 weights of 1 leaves room for one more below 2^64; the margins
// are larger.
__device__ __forceinline__ uint64_t add_up_to_most(uint64_t a, uint64_t b) { return a + b < a ? ~0ull : a + b; }

// Whether `left` lies inside [lo, hi) by more than `off`.
__device__ __forceinline__ bool well_inside(uint64_t lo, uint64_t left, uint64_t hi, uint64_t off) {
    return lo <= left && left < hi && left - lo >= off && hi - left > off;
}

// The nucleus' target mass, as the two ends of what it may be.
__device__ __forceinline__ void nucleus_target(const Ctrl* c, const ListRule& rule, uint64_t listed, uint64_t& lo,
                                               uint64_t& hi) {
    const uint64_t e = rule.complete ? 0 : c->margin, s = rule.complete ? listed : c->total;
    const float p = c->top_p;
    lo = p < 1.f ? scale_ceil(s - e, p) : ~0ull;
    hi = p < 1.f ? scale_ceil(add_up_to_most(s, e), p) : ~0ull;
}

// The row's token from a list of at most kThreads candidates, one thread each
// and no sort: a candidate's rank and the mass before it are sums over the
// list.  False when the list does not decide.
__device__ bool decide_small(const RowSearchArgs& a, const Smem& s, int n, ListRule rule, int64_t o) {
    Ctrl* c = s.c;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const uint64_t mine = t < n ? s.buf[t] : ~0ull;
    const uint64_t w = t < n ? weight44(candidate_value(mine), c->ws) : 0ull;
    if (t < n) s.wbuf[t] = w;
    __syncthreads();
    uint64_t before = 0;
    int rank = 0;
    if (t < n) {
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
            const bool less = s.buf[j] < mine;
            rank += less;
            before += less ? s.wbuf[j] : 0ull;
        }
    }
    const bool in_k = t < n && rank < rule.k;
    uint64_t listed;
    block_scan(in_k ? w : 0ull, c->scan, listed);
    uint64_t lo, hi;
    nucleus_target(c, rule, listed, lo, hi);
    const bool pass = in_k && w >= c->least;
    const bool stays = pass && before < hi;
    // bit 0: the nucleus ends inside the list, for every target it may have;
    // bit 1: a min-p token may lie past the nucleus' end; bit 2: min-p ends
    // inside the list
    int flags = (in_k && before < lo && before + w >= hi ? 1 : 0) | (pass && before >= lo ? 2 : 0) |
                (in_k && w < c->least ? 4 : 0);
    flags = __reduce_or_sync(DLM_FULL_MASK, flags);
    const int kept_here = __popc(__ballot_sync(DLM_FULL_MASK, stays));
    uint32_t first = __reduce_min_sync(DLM_FULL_MASK, stays ? (uint32_t)mine : 0xffffffffu);
    if (lane == 0) {
        c->hits[0][warp] = flags;
        c->hits[1][warp] = kept_here;
        c->first[warp] = first;
    }
    if (t < n) s.wbuf[t] = stays ? w : 0ull;
    uint64_t mass;
    block_scan(stays ? w : 0ull, c->scan, mass);
    flags = 0;
    int kept = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        flags |= c->hits[0][i];
        kept += c->hits[1][i];
        first = min(first, c->first[i]);
    }
    if (!rule.complete && !(flags & 1) && ((flags & 2) || !(rule.all_least || (flags & 4)))) return false;
    if (kept == 1) {
        if (stays) write_token(a, c, o, (int)(uint32_t)mine, candidate_value(mine), mass);
        return true;
    }
    if (stays) {
        bool cut;
        const uint64_t target = scale_floor(mass, c->u, cut);
        const uint32_t i = (uint32_t)mine;
        uint64_t run = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) run += (uint32_t)s.buf[j] < i ? s.wbuf[j] : 0ull;
        // u = 0: the first kept position, however small its weight
        if (c->u == 0.f ? i == first : (run <= target && target < run + w))
            write_token(a, c, o, (int)i, candidate_value(s.buf[t]), mass);
    }
    return true;
}

// How many of the n sorted candidates of a longer list stay (c->n, or -1 when
// the list does not decide), and their mass.
__device__ __noinline__ void keep_candidates(const Smem& s, int n, ListRule rule) {
    Ctrl* c = s.c;
    const int t = threadIdx.x, K = min(n, rule.k);
    const int per = (K + kThreads - 1) / kThreads, i0 = min(K, t * per), i1 = min(K, i0 + per);
    uint64_t sum = 0;
    for (int i = i0; i < i1; ++i) {
        const uint64_t w = weight_call(candidate_value(s.buf[i]), c->ws);
        s.wbuf[i] = w;
        sum += w;
    }
    if (t == 0) {
        c->n = c->top_p < 1.f ? -1 : K;
        c->batch = 0;
    }
    uint64_t listed;
    const uint64_t before = block_scan(sum, c->scan, listed);  // (its barriers order c->n too)
    uint64_t lo, hi;
    nucleus_target(c, rule, listed, lo, hi);
    // the nucleus: the shortest prefix whose mass reaches the target
    uint64_t m = before;
    int last = -1;
    for (int i = i0; i < i1; ++i) {
        const uint64_t w = s.wbuf[i];
        if (c->top_p < 1.f && m < lo && m + w >= hi) c->n = i + 1;
        // min-p keeps a prefix too, and the last token that passes ends it
        if (w >= c->least) last = i;
        m += w;
    }
    if (last >= 0) atomicMax(&c->batch, last + 1);
    __syncthreads();
    const int n_min = c->batch;
    // min-p ends the row when its last token surely belongs to the nucleus
    const bool inside = rule.complete || rule.all_least || n_min < K;
    bool by_min = false;
    m = before;
    for (int i = i0; i < i1; ++i) {
        by_min |= i == n_min - 1 && inside && m < lo;
        m += s.wbuf[i];
    }
    by_min = __syncthreads_or(by_min);
    if (t == 0 && by_min && (c->n < 0 || n_min < c->n)) c->n = n_min;
    __syncthreads();
    const int kept = c->n;
    m = before;
    for (int i = i0; i < i1; ++i) {
        m += s.wbuf[i];
        if (i == kept - 1) c->mass = m;
    }
    __syncthreads();
}

// The token among the first n candidates, in vocabulary order.
template <int DT>
__device__ __noinline__ void pick_candidate(const RowSearchArgs& a, const Smem& s, int n, const char* row, int64_t o) {
    Ctrl* c = s.c;
    const int t = threadIdx.x;
    const uint64_t mass = c->mass;
    bool cut;
    const uint64_t target = scale_floor(mass, c->u, cut);
    if (n == 1) {
        if (t == 0) write_token(a, c, o, (int)(uint32_t)s.buf[0], candidate_value(s.buf[0]), mass);
        return;
    }
    const bool first = c->u == 0.0f;  // the first kept position, however small its weight
    if (n <= kThreads) {
        if (t < n) {
            const uint32_t i = (uint32_t)s.buf[t];
            uint64_t before = 0;
            int less = 0;
            for (int j = 0; j < n; ++j) {
                const bool b = (uint32_t)s.buf[j] < i;
                before += b ? s.wbuf[j] : 0ull;
                less += b;
            }
            if (first ? less == 0 : (before <= target && target < before + s.wbuf[t]))
                write_token(a, c, o, (int)i, candidate_value(s.buf[t]), mass);
        }
        return;
    }
    for (int i = t; i < n; i += kThreads) s.buf[i] = (s.buf[i] << 32) | (uint32_t)i;
    __syncthreads();
    constexpr int kRoom = kCap - kSortBins / 2;  // (bins behind the weights)
    sort_u64(s.buf, n, n <= kRoom ? s.wbuf + kRoom : nullptr, c);
    const int per = (n + kThreads - 1) / kThreads, i0 = min(n, t * per), i1 = min(n, i0 + per);
    uint64_t sum = 0, total;
    for (int i = i0; i < i1; ++i) sum += s.wbuf[(uint32_t)s.buf[i]];
    uint64_t m = block_scan(sum, c->scan, total);
    for (int i = i0; i < i1; ++i) {
        const uint64_t next = m + s.wbuf[(uint32_t)s.buf[i]];
        if (first ? i == 0 : (m <= target && target < next)) write_token(a, c, o, (int)(s.buf[i] >> 32), Row<DT>::scalar(row, (int64_t)(s.buf[i] >> 32)), mass);
        m = next;
    }
}

// ---- the search over the whole row ----------------------------------------
// Every CTA of the cluster works its batches; the first one merges.

// One radix pass over the keys of a slice: bin b of the kBins gets the count
// (MASS false) or the mass (true) of the elements whose key has the bits
// `prefix` above shift + 11 and b below.  lo / hi: the two 32-bit halves.
template <int DT, bool MASS>
__device__ __noinline__ void radix_pass(const char* row, int64_t V, int b0, int b1, uint32_t prefix, int shift, int bits,
                           uint32_t floor_key, const WeightScale& ws, uint32_t* lo, uint32_t* hi) {
    constexpr int EPV = Row<DT>::EPV;
    for (int i = threadIdx.x; i < kBins; i += kThreads) lo[i] = hi[i] = 0;
    __syncthreads();
    const uint32_t mask = (1u << bits) - 1u;
    for (int v = b0 * kBatchVecs + (int)threadIdx.x; v < b1 * kBatchVecs; v += kThreads) {
        float z[EPV];
        Row<DT>::unpack(load_vec<DT>(row, V, v), z);
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
            const uint32_t key = key_of(z[e]);
            if (key <= floor_key || (shift + bits < 32 && (key >> (shift + bits)) != prefix)) continue;
            const uint32_t bin = (key >> shift) & mask;
            if constexpr (MASS) {
                const uint64_t w = weight_call(z[e], ws);
                const uint32_t wl = (uint32_t)w;
                const uint32_t old = atomicAdd(&lo[bin], wl);
                const uint32_t up = (uint32_t)(w >> 32) + (old + wl < old ? 1u : 0u);
                if (up) atomicAdd(&hi[bin], up);
            } else {
                atomicAdd(&lo[bin], 1u);
            }
        }
    }
    __syncthreads();
}

// The bin in which the running sum from the top, starting at `above`, first
// reaches `target`, over the cluster's merged bins.  Returns through the first
// CTA's ctrl: prefix (with the bin appended), above (before the bin), and
// total (the sum of all bins) -- left unchanged but for total when no bin
// reaches it.  kThreads threads, kBins / kThreads bins each.
__device__ __noinline__ void radix_pick(const Cluster& cl, const Smem& s, uint32_t prefix, int bits, uint64_t above,
                           uint64_t target) {
    cl.sync();
    if (cl.rank == 0) {
        constexpr int PER = kBins / kThreads;
        uint32_t* lo = reinterpret_cast<uint32_t*>(s.buf);
        uint32_t* hi = lo + kBins;
        uint64_t v[PER], sum = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int bin = kBins - 1 - ((int)threadIdx.x * PER + j);
            uint64_t x = 0;
            for (int r = 0; r < cl.split; ++r)
                x += ((uint64_t)cl.at(hi, r)[bin] << 32) + cl.at(lo, r)[bin];
            v[j] = x;
            sum += x;
        }
        uint64_t total;
        uint64_t m = above + block_scan(sum, s.c->scan, total);
        if (threadIdx.x == 0) s.c->total = total;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int bin = kBins - 1 - ((int)threadIdx.x * PER + j);
            if (m < target && target <= m + v[j]) {
                s.c->prefix = (prefix << bits) | (uint32_t)bin;
                s.c->above = m;
                s.c->mass = v[j];
            }
            m += v[j];
        }
    }
    cl.sync();
}

// A key's 32 bits in three passes: 11, 11 and 10.
__device__ __forceinline__ int radix_shift(int l) { return l == 0 ? 21 : l == 1 ? 10 : 0; }
__device__ __forceinline__ int radix_bits(int l) { return l == 2 ? 10 : 11; }

// Top-k over the whole row: the k-th key of the order and how many positions
// at it belong to the k (fewer finite logits than k: every one of them).
// When the keys at or above a bin fit the candidate list the search stops
// there: *list is set and the result is that bin's lower edge.
template <int DT>
__device__ __noinline__ void count_cut(const Cluster& cl, const Smem& s, const char* row, int64_t V, int b0, int b1, int k,
                          const WeightScale& ws, uint32_t& key, uint32_t& ties, bool& list) {
    uint32_t* lo = reinterpret_cast<uint32_t*>(s.buf);
    const Ctrl* c0 = cl.at(s.c, 0);
    uint32_t prefix = 0;
    uint64_t above = 0;
    list = false;
    for (int l = 0; l < 3; ++l) {
        radix_pass<DT, false>(row, V, b0, b1, prefix, radix_shift(l), radix_bits(l), kKeyNegInf, ws, lo, lo + kBins);
        radix_pick(cl, s, prefix, radix_bits(l), above, (uint64_t)k);
        if (l == 0 && c0->total < (uint64_t)k) {  // fewer finite logits: all of them
            list = c0->total <= (uint64_t)kCap;
            // (no ties at the lowest float: their number is not known, and where it is
            // the maximum their weight is 1)
            key = list ? kKeyNegInf + 1 : kKeyNegInf;
            ties = 0;
            cl.sync();
            return;
        }
        prefix = c0->prefix;
        above = c0->above;
        const uint64_t up_to = above + c0->mass;
        cl.sync();
        if (up_to <= (uint64_t)kCap) {
            list = true;
            key = max(prefix << radix_shift(l), kKeyNegInf + 1);
            ties = 0xffffffffu;
            return;
        }
    }
    key = prefix;
    ties = (uint32_t)((uint64_t)k - above);
}

// Top-p over the keys above floor_key plus floor_ties positions at it: the
// key at which the mass reaches p of the total, and how many positions there.
template <int DT>
__device__ __noinline__ void mass_cut(const Cluster& cl, const Smem& s, const char* row, int64_t V, int b0, int b1, float p,
                         uint32_t floor_key, uint32_t floor_ties, const WeightScale& ws, uint32_t& key,
                         uint32_t& ties) {
    uint32_t* lo = reinterpret_cast<uint32_t*>(s.buf);
    const Ctrl* c0 = cl.at(s.c, 0);
    const uint64_t w_floor = floor_key > kKeyNegInf ? weight_call(key_value(floor_key), ws) : 0;
    uint32_t prefix = 0;
    uint64_t above = 0, target = ~0ull, total = 0;
    for (int l = 0; l < 3; ++l) {
        radix_pass<DT, true>(row, V, b0, b1, prefix, radix_shift(l), radix_bits(l), floor_key, ws, lo, lo + kBins);
        if (l == 0) {
            // the total first (no bin can reach an unreachable target)
            radix_pick(cl, s, 0, radix_bits(0), 0, ~0ull);
            total = c0->total;
            target = scale_ceil(total + w_floor * floor_ties, p);
            cl.sync();
            if (target > total) {  // it ends among the ties of the top-k's last key
                key = floor_key;
                ties = w_floor ? (uint32_t)min((uint64_t)floor_ties, (target - total + w_floor - 1) / w_floor)
                               : floor_ties;
                return;
            }
        }
        radix_pick(cl, s, prefix, radix_bits(l), above, target);
        prefix = c0->prefix;
        above = c0->above;
        cl.sync();
    }
    key = prefix;
    const uint64_t w = weight_call(key_value(key), ws);  // > 0: its bin had mass
    ties = (uint32_t)((target - above + w - 1) / w);
}

// Mass of the keys above cut_key with a weight of at least `least`, and the
// number of positions at cut_key, per batch.
template <int DT>
__device__ __noinline__ void batch_masses(const char* row, int64_t V, int b0, int b1, uint32_t cut_key, uint64_t least,
                                          const WeightScale& ws, uint64_t* bmass, uint32_t* bties) {
    constexpr int EPV = Row<DT>::EPV;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int b = b0 + warp; b < b1; b += kWarps) {
        uint64_t m = 0;
        int ties = 0;
        for (int i = 0; i < kRuns; ++i) {
            float z[EPV];
            Row<DT>::unpack(load_vec<DT>(row, V, b * kBatchVecs + i * 32 + lane), z);
#pragma unroll
            for (int e = 0; e < EPV; ++e) {
                const uint32_t key = key_of(z[e]);
                if (key > cut_key) {
                    const uint64_t w = weight_call(z[e], ws);
                    m += w >= least ? w : 0ull;
                }
                ties += key == cut_key;
            }
        }
        m = (uint64_t)warp_sum_ll((long long)m);
        ties = warp_sum_i(ties);
        if (lane == 0) {
            bmass[b] = m;
            bties[b] = (uint32_t)ties;
        }
    }
}

// The batch that holds the target, among nb batches in order; the kept ties
// of a batch are those whose rank over the row is below cut_ties.  Sets ctrl:
// mass (all kept), batch, left (target inside it), ties_before.
__device__ void find_batch(const Smem& s, int nb, uint64_t w_tie, uint32_t cut_ties) {
    Ctrl* c = s.c;
    const int t = threadIdx.x;
    const int per = (nb + kThreads - 1) / kThreads, b0 = min(nb, t * per), b1 = min(nb, b0 + per);
    uint64_t ties0 = 0;
    if (w_tie) {
        uint64_t n = 0, total;
        for (int b = b0; b < b1; ++b) n += s.bties[b];
        ties0 = block_scan(n, c->scan, total);
    }
    auto tie_mass = [&](int b, uint64_t& ties) {
        if (!w_tie) return (uint64_t)0;
        const uint64_t room = ties < cut_ties ? cut_ties - ties : 0;
        ties += s.bties[b];
        return min((uint64_t)s.bties[b], room) * w_tie;
    };
    uint64_t ties = ties0, m = 0;
    for (int b = b0; b < b1; ++b) m += s.bmass[b] + tie_mass(b, ties);
    uint64_t mass;
    uint64_t before = block_scan(m, c->scan, mass);
    bool cut;
    const uint64_t target = scale_floor(mass, c->u, cut);
    ties = ties0;
    for (int b = b0; b < b1; ++b) {
        const uint32_t ties_here = (uint32_t)ties;
        const uint64_t here = s.bmass[b] + tie_mass(b, ties);
        if (before <= target && target < before + here) {
            c->batch = b;
            c->left = target - before;
            c->ties_before = ties_here;
        }
        before += here;
    }
    if (t == 0) c->mass = mass;
    __syncthreads();
}

// The whole CTA walks the chosen batch (ctrl: batch, left, cut_key, cut_ties,
// cut_last, ties_before, least) to the element whose running kept mass passes
// `left`: in ctrl, its position (token, -1 if there is none) and the sums on
// both sides of it (lo_side, hi_side).  A thread takes 8 bytes of the batch.
template <int DT>
__device__ __noinline__ void walk_batch(const char* row, int64_t V, Ctrl* c) {
    constexpr int N = 8 / Row<DT>::ESZ;
    static_assert(N * kThreads == kBatchVecs * Row<DT>::EPV, "a batch is 8 bytes per thread");
    const int t = threadIdx.x;
    const int64_t at = (int64_t)c->batch * (N * kThreads) + t * N;
    const uint32_t cut_key = c->cut_key, cut_ties = c->cut_ties;
    const WeightScale ws = c->ws;
    float z[N];
#pragma unroll
    for (int e = 0; e < N; ++e) z[e] = at + e < V ? Row<DT>::scalar(row, at + e) : -INFINITY;
    if (t == 0) c->token = -1;
    uint64_t rank = 0, sum = 0, all;
    if (cut_ties != 0 && cut_ties != 0xffffffffu) {  // a tie's rank over the row decides
        uint64_t mine = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) mine += key_of(z[e]) == cut_key;
        rank = c->ties_before + block_scan(mine, c->scan, all);
    }
    uint64_t w[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const uint32_t key = key_of(z[e]);
        const bool tie = key == cut_key;
        const bool stays = key > cut_key || (tie && rank < cut_ties && (uint32_t)(at + e) <= c->cut_last);
        w[e] = stays ? weight_call(z[e], ws) : 0ull;
        if (w[e] < c->least) w[e] = 0;
        rank += tie;
        sum += w[e];
    }
    uint64_t m = block_scan(sum, c->scan, all);
    const uint64_t left = c->left;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        if (m <= left && left < m + w[e]) {
            c->token = (int)(at + e);
            c->z = z[e];
            c->lo_side = m;
            c->hi_side = m + w[e];
        }
        m += w[e];
    }
    __syncthreads();
}

// u = 0: the first kept position of the row, whatever its weight (one warp of
// the first CTA; reads the row until it meets one).
template <int DT>
__device__ __noinline__ int first_kept(const char* row, int64_t V, int nb, const Ctrl* c) {
    constexpr int EPV = Row<DT>::EPV;
    const int lane = threadIdx.x & 31;
    const WeightScale ws = c->ws;
    for (int v0 = 0; v0 < nb * kBatchVecs; v0 += 32) {
        float z[EPV];
        Row<DT>::unpack(load_vec<DT>(row, V, v0 + lane), z);
        int e0 = EPV;
#pragma unroll
        for (int e = EPV - 1; e >= 0; --e) {
            const uint32_t key = key_of(z[e]);
            const bool in = key > c->cut_key || (key == c->cut_key && c->cut_ties > 0 &&
                                                 (uint32_t)((v0 + lane) * EPV + e) <= c->cut_last);
            if (in && (c->least == 0 || weight_call(z[e], ws) >= c->least)) e0 = e;
        }
        const uint32_t who = __ballot_sync(DLM_FULL_MASK, e0 < EPV);
        if (who) {
            const int src = __ffs(who) - 1;
            return (v0 + src) * EPV + __shfl_sync(DLM_FULL_MASK, e0, src);
        }
    }
    return -1;
}

// ---- the nucleus by a bracket ------------------------------------------------

// Two weights in 32 bits with a relative error below 6 * 2^-24: the exponent's
// integer part goes into the float's exponent field exactly, ex2 sees the
// fraction.  The logits must be within 100 powers of 2 of the maximum.
struct SplitScale {
    f2 m, nc_hi, nc_lo;  // the maximum, and minus log2(e) / T in two floats
};
__device__ __forceinline__ f2 weight_split(f2 z, const SplitScale& s) {
    const f2 magic = pack2(12582912.0f, 12582912.0f);  // 1.5 * 2^23: rounds to an integer
    const f2 d = sub2(s.m, z);
    const f2 b = sub2(d, s.m);
    const f2 err = sub2(sub2(s.m, sub2(d, b)), add2(z, b));
    const f2 t = fma2(d, s.nc_hi, magic);
    f2 f = fma2(d, s.nc_hi, sub2(magic, t));
    f = fma2(d, s.nc_lo, f);
    f = fma2(err, s.nc_hi, f);
    float x, y, tx, ty;
    unpack2(ex2x2(f), x, y);
    unpack2(t, tx, ty);
    return pack2(__int_as_float(__float_as_int(x) + (__float_as_int(tx) << 23)),
                 __int_as_float(__float_as_int(y) + (__float_as_int(ty) << 23)));
}

// Two weights as T 2^-n + a correction in 32 bits: 32 y = k + r, T = 2^(-j / 32)
// with j = k mod 32, n = k div 32, T = table value M 2^-24 + lo exactly, so the
// weight is (M << 20) >> n in units of 2^-44 plus (M 2^-24 (2^(-r / 32) - 1) + lo)
// 2^-n, whose error is below 2^-28 of the weight.  `tab`: this lane's column of
// the 32 values as floats M 2^-24, `tab + 1024` of the lo (a copy per bank).
struct FineScale {
    f2 m, nc_hi, nc_lo;  // the maximum, and minus 32 log2(e) / T in two floats
    const float* tab;
};
__device__ __forceinline__ void weight_fine(f2 z, const FineScale& s, uint64_t (&hi)[2], f2& lo) {
    const f2 magic = pack2(12582912.0f, 12582912.0f);
    const f2 d = sub2(s.m, z);
    const f2 b = sub2(d, s.m);
    const f2 err = sub2(sub2(s.m, sub2(d, b)), add2(z, b));
    const f2 t = fma2(d, s.nc_hi, magic);  // magic - k
    f2 f = fma2(d, s.nc_hi, sub2(magic, t));
    f = fma2(d, s.nc_lo, f);
    f = fma2(err, s.nc_hi, f);
    const f2 x = mul2(f, pack2(0.021660849392498291f, 0.021660849392498291f));  // ln 2 / 32
    // e^x - 1 = x + x^2 / 2 + x^3 / 6 + x^4 / 24, |x| < 0.011
    f2 q = fma2(x, pack2(1.f / 24, 1.f / 24), pack2(1.f / 6, 1.f / 6));
    q = fma2(q, x, pack2(0.5f, 0.5f));
    q = fma2(q, x, pack2(1.f, 1.f));
    q = mul2(q, x);
    float tt[2], qq[2], l[2];
    unpack2(t, tt[0], tt[1]);
    unpack2(q, qq[0], qq[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int k = 0x4b400000 - __float_as_int(tt[i]), j = k & 31, n = k >> 5;
        const float v = s.tab[j * 32];
        const uint32_t m = (__float_as_uint(v) & 0x7fffffu) | 0x800000u;  // v is in [1/2, 1)
        hi[i] = ((uint64_t)m << 20) >> n;
        l[i] = fmaf(v, qq[i], s.tab[1024 + j * 32]) * __int_as_float((127 - n) << 23);
    }
    lo = pack2(l[0], l[1]);
}

// The smallest logit that min-p can keep (or one a little lower: the weights
// decide).
__device__ __forceinline__ float min_p_logit(const Ctrl* c) {
    return c->ws.m + (1.0001f * __logf(c->min_p) - 1e-5f) / (c->ws.c_hi * kLn2) - 1e-6f * fabsf(c->ws.m);
}

// The cluster's bins added up in the first CTA: each CTA takes its share of them.
// (By the first CTA alone, 32 remote loads per thread for a bracket's, 32 rows of
// 126464 take 57.6 us instead of 55.5.)
template <typename T>
__device__ __noinline__ void merge_bins(const Cluster& cl, T* bins, int n) {
    const int per = n / cl.split;
    for (int i = cl.rank * per + (int)threadIdx.x; i < (cl.rank + 1) * per; i += kThreads) {
        T v[8], sum = 0;
#pragma unroll
        for (int rk = 0; rk < 8; ++rk) v[rk] = rk < cl.split ? cl.at(bins, rk)[i] : 0;
#pragma unroll
        for (int rk = 0; rk < 8; ++rk) sum += v[rk];
        cl.at(bins, 0)[i] = sum;
    }
}

// A sample of `tokens` of the row in buf's kBins words: per 1/32 of an exponent below the
// maximum the weights relative to the bin's upper end, in 2^-16 (between 0.97
// and 1 each, so the bin counts its tokens too).  Returns how many of the row's
// tokens one of the sample stands for.
// The cluster's CTAs take a share each (merge_bins adds them up).
template <int DT>
__device__ __noinline__ float sample_row(const Cluster& cl, const char* row, int64_t V, const Smem& s, int tokens,
                                         float m, float c_hi) {
    constexpr int EPV = Row<DT>::EPV;
    const int t = threadIdx.x, lane = t & 31, warps = kWarps * cl.split, warp = cl.rank * kWarps + (t >> 5);
    uint32_t* bins = reinterpret_cast<uint32_t*>(s.buf);
    for (int i = t; i < kBins; i += kThreads) bins[i] = 0;
    __syncthreads();
    const int nsub = (int)((V + 32 * EPV - 1) / (32 * EPV));
    const int n = min(nsub, tokens / (32 * EPV));
    const float c32 = c_hi * 32.f;
    const int stride = nsub / n;
    auto fetch = [&](int i) { return i < n ? load_vec<DT>(row, V, i * stride * 32 + lane) : make_uint4(0, 0, 0, 0); };
    uint4 w0 = fetch(warp), w1 = fetch(warp + warps), w2 = fetch(warp + 2 * warps);
#pragma unroll 1
    for (int i = warp; i < n; i += warps) {
        float z[EPV];
        Row<DT>::unpack(w0, z);
        w0 = w1;
        w1 = w2;
        w2 = fetch(i + 3 * warps);
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
            if (!(z[e] > -INFINITY)) continue;
            const float x = (m - z[e]) * c32;
            const int bin = min(kBins - 1, (int)x);
            atomicAdd(&bins[bin], (uint32_t)(65536.f * ex2(fmaxf(((float)bin - x) * 0.03125f, -1.f))));
        }
    }
    __syncthreads();
    return (float)nsub / (float)n;
}

// Two logits that the nucleus' end should lie between: the mass below it is
// (1 - top_p) of the total, the sample tells where the row's lower end adds up
// to that, and the bracket takes the kBracketSide tokens on either side.  On a
// flat row of 152064 tokens that is three to four standard deviations of the
// sample; where few tokens hold the mass it reaches up to the largest.  When
// min-p's cut is higher the bracket is put around it.  `scale`: how many tokens one
// of the sample stands for.  One CTA; sets c->bin_lo, c->bin_hi and returns
// kTier1 or kMinP.
__device__ __noinline__ int place_bracket(const Smem& s, float scale) {
    constexpr int PER = kBins / kThreads;
    const int t = threadIdx.x;
    Ctrl* c = s.c;
    const uint32_t* bins = reinterpret_cast<const uint32_t*>(s.buf);
    const bool by_least = c->least > 0;
    const int cut = by_least ? (int)fminf((c->ws.m - min_p_logit(c)) * c->ws.c_hi * 32.f, (float)(kBins - 2)) : kBins;
    float want = 0.f;
    if (t == 0) {  // for a sample that does not reach it
        c->left = 0;
        c->bin_lo = kBins;
        c->bin_hi = 0;
        c->batch = kBins;
    }
    if (c->top_p < 1.f) {
        // thread t takes bins from the lowest weights up
        float mass = 0.f;
        uint64_t tokens = 0;  // in 2^-16, a little short
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int bin = kBins - 1 - (t * PER + j);
            mass += (float)bins[bin] * 0x1p-16f * ex2(-(float)bin * 0.03125f);
            tokens += bins[bin];
        }
        // exclusive sums over the threads in integers (a sample's mass is at most 2^14)
        uint64_t all;
        float run = (float)block_scan((uint64_t)__float2ull_rn(mass * 0x1p44f), c->scan, all) * 0x1p-44f;
        const uint64_t seen0 = block_scan(tokens, c->scan, all);
        uint64_t seen = seen0;
        // the sample's share of the mass below the nucleus' end
        want = (1.f - c->top_p) * ((float)c->total * 0x1p-44f) / scale;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int bin = kBins - 1 - (t * PER + j);
            const float next = run + (float)bins[bin] * 0x1p-16f * ex2(-(float)bin * 0.03125f);
            if (run <= want && next > want) {
                c->left = seen + bins[bin] / 2;
                c->batch = bin;
            }
            run = next;
            seen += bins[bin];
        }
        __syncthreads();
        const uint64_t mid = c->left, side = (uint64_t)((float)kBracketSide * 65536.f / scale);
        seen = seen0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int bin = kBins - 1 - (t * PER + j);
            const uint64_t next = seen + bins[bin];
            if (mid > side && seen <= mid - side && next > mid - side) c->bin_lo = bin + 1;
            if (seen < mid + side && next >= mid + side) c->bin_hi = bin;
            seen = next;
        }
    }
    __syncthreads();
    const bool by_min = by_least && cut <= c->batch;
    __syncthreads();
    if (t == 0 && by_min) {
        c->bin_lo = cut + 2;
        c->bin_hi = max(cut - 1, 0);
    }
    __syncthreads();
    return by_min ? kMinP : kTier1;
}

// A threshold that about sqrt(k kCap) of the row's logits reach, between k and
// the list's length by three standard deviations of the sample.  One CTA; sets
// c->bin_lo and returns kList, or kRadix when no bin is near.
__device__ __noinline__ int place_list(int k, const Smem& s, float scale) {
    constexpr int PER = kBins / kThreads;
    const int t = threadIdx.x;
    Ctrl* c = s.c;
    const uint32_t* bins = reinterpret_cast<const uint32_t*>(s.buf);
    if (t == 0) c->bin_lo = 0;
    uint64_t tokens = 0, all;
#pragma unroll
    for (int j = 0; j < PER; ++j) tokens += bins[t * PER + j];
    uint64_t seen = block_scan(tokens, c->scan, all);  // from the largest down
    const float want = sqrtf((float)k * (float)kCap) * 64700.f / scale;  // a token counts 0.987 * 2^16 on average
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const uint64_t next = seen + bins[t * PER + j];
        if ((float)seen < want && (float)next >= want) c->bin_lo = t * PER + j + 1;
        seen = next;
    }
    __syncthreads();
    return c->bin_lo > 0 && c->bin_lo < kBins ? kList : kRadix;
}

// The bracket in logits from its bins (one thread).
__device__ __forceinline__ void set_bracket(Ctrl* c, int verdict) {
    const float c32 = c->ws.c_hi * 32.f;
    c->z_lo = c->ws.m - (float)c->bin_lo / c32;
    c->z_hi = c->ws.m - (float)c->bin_hi / c32;
    c->by_min = verdict == kMinP;
    if (verdict == kTier1 && c->top_p >= 1.f) c->z_lo = c->z_hi = -INFINITY;  // everything is above: sums only
    c->tries = 0;
}

// One pass over a slice: bmass[b] the mass of batch b at z >= z_hi, c->whole
// the slice's whole mass, and the tokens of [z_lo, z_hi) into dst, c->count of
// them (which may exceed kBracketCap).  TIER 1: weight_split summed over a vector
// in 32 bits, 2: weight_fine (its table in `fine`), 3: integer weights.
template <int DT, int TIER>
__device__ __noinline__ void bracket_pass(const char* row, int64_t V, int b0, int b1, float z_lo, float z_hi,
                                          const WeightScale ws, uint64_t* bmass, Ctrl* c, uint64_t* dst,
                                          float* fine) {
    constexpr int EPV = Row<DT>::EPV;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // a weight of 2^-60 counts as 0
    const float z_min = fmaxf(ws.m - 60.f / ws.c_hi, -FLT_MAX), c32 = -32.f * ws.c_hi, d32 = -32.f * ws.c_lo;
    const SplitScale sp{pack2(ws.m, ws.m), pack2(-ws.c_hi, -ws.c_hi), pack2(-ws.c_lo, -ws.c_lo)};
    const FineScale fs{pack2(ws.m, ws.m), pack2(c32, c32), pack2(d32, d32), fine + lane};
    if (TIER == 2) {
        for (int i = threadIdx.x; i < 1024; i += kThreads) {
            const uint64_t v = ws.tab[(i >> 5) * 8];
            const uint32_t m = min((uint32_t)(v >> 20), 0xffffffu);
            fine[i] = (float)m * 0x1p-24f;
            fine[1024 + i] = (float)(uint32_t)(v - ((uint64_t)m << 20)) * 0x1p-44f;
        }
        __syncthreads();
    }
    uint64_t whole = 0, top = 0, sum = 0;
    // a run at a time (one copy of the code), two more on their way: the warp's
    // i-th run is run i % 4 of its batch i / 4
    const int runs = b0 + warp < b1 ? ((b1 - b0 - warp + kWarps - 1) / kWarps) * kRuns : 0;
    auto vec_of = [&](int i) { return ((b0 + warp + (i / kRuns) * kWarps) * kRuns + i % kRuns) * 32 + lane; };
    auto fetch = [&](int i) { return i < runs ? load_vec<DT>(row, V, vec_of(i)) : make_uint4(0, 0, 0, 0); };
    uint4 w1 = fetch(0), w2 = fetch(1);
    uint64_t above = 0;
#pragma unroll 1
    for (int i = 0; i < runs; ++i) {
        const uint4 w0 = w1;
        w1 = w2;
        w2 = fetch(i + 2);
        float z[EPV];
        Row<DT>::unpack(w0, z);
        uint32_t mask = 0;  // tokens inside, a bit each
        if constexpr (TIER == 3) {
#pragma unroll
            for (int e = 0; e < EPV; ++e) {
                const uint64_t w = weight_call(z[e], ws);
                const bool up = z[e] >= z_hi;
                above += up ? w : 0ull;
                whole += w;
                mask |= (uint32_t)(!up && z[e] >= z_lo) << e;
            }
        } else if constexpr (TIER == 2) {
            f2 up = pack2(0.f, 0.f), all = pack2(0.f, 0.f);
#pragma unroll
            for (int p = 0; p < EPV / 2; ++p) {
                const float x = fmaxf(z[2 * p], z_min), y = fmaxf(z[2 * p + 1], z_min);
                uint64_t w[2];
                f2 lo;
                weight_fine(pack2(x, y), fs, w, lo);
                const bool ux = x >= z_hi, uy = y >= z_hi;
                above += (ux ? w[0] : 0ull) + (uy ? w[1] : 0ull);
                whole += w[0] + w[1];
                float lx, ly;
                unpack2(lo, lx, ly);
                all = add2(all, lo);
                up = add2(up, pack2(ux ? lx : 0.f, uy ? ly : 0.f));
                mask |= (uint32_t)(!ux && x >= z_lo) << (2 * p);
                mask |= (uint32_t)(!uy && y >= z_lo) << (2 * p + 1);
            }
            above += (uint64_t)__float2ll_rn(hsum2(up) * 0x1p44f);
            whole += (uint64_t)__float2ll_rn(hsum2(all) * 0x1p44f);
        } else {
            f2 up[EPV / 2], all[EPV / 2];
#pragma unroll
            for (int p = 0; p < EPV / 2; ++p) {
                const float x = fmaxf(z[2 * p], z_min), y = fmaxf(z[2 * p + 1], z_min);
                all[p] = weight_split(pack2(x, y), sp);
                float wx, wy;
                unpack2(all[p], wx, wy);
                const bool ux = x >= z_hi, uy = y >= z_hi;
                up[p] = pack2(ux ? wx : 0.f, uy ? wy : 0.f);
                mask |= (uint32_t)(!ux && x >= z_lo) << (2 * p);
                mask |= (uint32_t)(!uy && y >= z_lo) << (2 * p + 1);
            }
#pragma unroll
            for (int h = EPV / 4; h; h >>= 1)
#pragma unroll
                for (int p = 0; p < h; ++p) {
                    up[p] = add2(up[p], up[p + h]);
                    all[p] = add2(all[p], all[p + h]);
                }
            above += __float2ull_rn(hsum2(up[0]) * 0x1p44f);
            whole += __float2ull_rn(hsum2(all[0]) * 0x1p44f);
        }
        if (i % kRuns == kRuns - 1) {
            top += above;
            above = (uint64_t)warp_sum_ll((long long)above);
            if (lane == 0) bmass[b0 + warp + (i / kRuns) * kWarps] = above;
            above = 0;
        }
        if (!__any_sync(DLM_FULL_MASK, mask != 0)) continue;
        const int mine = __popc(mask);
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(DLM_FULL_MASK, inc, o);
            if (lane >= o) inc += x;
        }
        uint32_t at = 0;
        if (lane == 31) at = atomicAdd(&c->count, (uint32_t)inc);
        at = __shfl_sync(DLM_FULL_MASK, at, 31) + (uint32_t)(inc - mine);
#pragma unroll
        for (int e = 0; e < EPV; ++e)
            if ((mask >> e) & 1u) {
                if (at < (uint32_t)kBracketCap) dst[at] = candidate(z[e], (uint32_t)(vec_of(i) * EPV + e));
                ++at;
            }
    }
    block_scan(whole, c->scan, sum);
    if (threadIdx.x == 0) c->whole = sum;
    block_scan(top, c->scan, sum);
    if (threadIdx.x == 0) c->top = sum;
    __syncthreads();
}

// The bin of a bracket's token, from z_hi down.
__device__ __forceinline__ int fine_bin(uint64_t e, float z_hi, float per_bin) {
    return max(0, min(kFine - 1, (int)((z_hi - candidate_value(e)) * per_bin)));
}

// A slice's tokens of the bracket into its CTA's bins, with their mass.  16-bit
// logits repeat: equal ones of a warp are added once.
__device__ __noinline__ void bin_tokens(const Smem& s, float z_hi, float per_bin, const WeightScale ws) {
    const int t = threadIdx.x, n = (int)min(s.c->count, (uint32_t)kBracketCap);
    for (int i = t; i < kFine; i += kThreads) s.fine[i] = 0;
    __syncthreads();
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + t;
        const uint64_t e = i < n ? s.buf[i] : 0;
        const uint32_t like = __match_any_sync(DLM_FULL_MASK, i < n ? (uint32_t)(e >> 32) : 0xffffffffu);
        if (i < n && __ffs(like) - 1 == (t & 31))
            shared_add(&s.fine[fine_bin(e, z_hi, per_bin)], weight_call(candidate_value(e), ws) * __popc(like));
    }
    __syncthreads();
}

// After a pass, in the first CTA: where the row ends.  Every weight of the
// pass is off by the share err / total at most, so a sum over part of the mass
// and that part's share of the whole differ by 2 share (1 - share) err at most
// from what they should.  Returns kDone when the end is inside the bracket:
// ctrl then has the bins that may hold it (first_bin, last_bin), the mass before
// them (left) and the targets; else another bracket is set and it is a tier's,
// or kRadix.
__device__ __noinline__ int find_end(const Cluster& cl, const Smem& s, int nb, int tier) {
    Ctrl* c = s.c;
    const int t = threadIdx.x;
    uint64_t total = 0, above = 0, n = 0;
#pragma unroll
    for (int rk = 0; rk < 8; ++rk) {
        if (rk >= cl.split) break;
        const Ctrl* rc = cl.at(c, rk);
        total += rc->whole;
        above += rc->top;
        n = max(n, (uint64_t)rc->count);
    }
    // tier 1, in 2^-24: ex2 4, the fraction's roundings and the conversion 2,
    // three levels of additions 3.  Tier 2, in 2^-24 of a correction that is at
    // most 2^-6.5 of its weight: the table's product 2, the power 2, the
    // exponent's roundings 2, additions 4.  Tier 3: integer weights, 2^-37
    const uint64_t err = (tier == kTier1 ? (total >> 24) * 9 : total >> (tier == kTier2 ? 27 : 36)) + 4 * (uint64_t)nb;
    const float p = c->top_p;
    const uint64_t x = p < 1.f ? scale_ceil(total, p) : ~0ull;
    const uint64_t off = p < 1.f ? (uint64_t)((float)err * 2.0001f * p * (1.f - p)) + 2 : 0;  // rounded up
    // another bracket: above this one or below (with a quarter of it), the
    // middle of one that holds too many tokens, or min-p's
    enum { kUp, kDown, kMiddle, kToMin };
    auto miss = [&](int how) {
        __syncthreads();
        if (t == 0) {
            const float lo = c->z_lo, hi = c->z_hi, width = fmaxf(hi - lo, 1e-6f * fabsf(hi));
            if (how == kUp) {
                c->z_lo = hi - 0.25f * width;
                c->z_hi = hi + 2.f * width;
            } else if (how == kDown) {
                c->z_lo = lo - 2.f * width;
                c->z_hi = lo + 0.25f * width;
            } else if (how == kMiddle) {
                c->z_lo = lo + 0.4f * width;
                c->z_hi = hi - 0.4f * width;
            } else {
                const float z = min_p_logit(c), step = 0.03125f / c->ws.c_hi;
                c->z_lo = z - step;
                c->z_hi = z + step;
                c->by_min = 1;
            }
            c->tries += 1;
        }
        __syncthreads();
        return c->tries < kTries ? tier : (int)kRadix;
    };
    if (t == 0) {
        c->total = total;
        c->err = err;
        c->runs = 0;
        c->above = above;
    }
    if (c->by_min) {
        if (n > (uint64_t)kBracketCap) return kRadix;
        // the cut has to be inside the bracket (the logits' estimate was near)
        if (weight_call(fminf(c->z_hi, c->ws.m), c->ws) < c->least || weight_call(c->z_lo, c->ws) >= c->least) return kRadix;
        __syncthreads();
        return kDone;
    }
    if (p >= 1.f) {
        __syncthreads();
        return kDone;
    }
    // what is above is short of the target, what is above and inside reaches
    // it, and all of it is listed
    if (above + off >= x) return miss(kUp);
    if (n > (uint64_t)kBracketCap) return miss(kMiddle);
    const uint64_t t_lo = x - above - off, t_hi = x - above + off;
    constexpr int PER = kFine / kThreads;
    uint64_t v[PER], sum = 0, inside;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        v[j] = s.fine[t * PER + j];
        sum += v[j];
    }
    uint64_t m = block_scan(sum, c->scan, inside);
    if (inside < t_hi) return miss(kDown);
    if (t == 0) {
        c->t_lo = t_lo;
        c->t_mid = x - above;
        c->t_hi = t_hi;
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const uint64_t next = m + v[j];
        if (m < t_lo && next >= t_lo) {
            c->first_bin = t * PER + j;
            c->left = m;
        }
        if (m < t_hi && next >= t_hi) c->last_bin = t * PER + j;
        m = next;
    }
    __syncthreads();
    // (a bin's lowest logit, and what else is in it, decides min-p)
    if (c->least > 0) {
        const float z = c->z_hi - (float)(c->last_bin + 1) / (float)kFine * (c->z_hi - c->z_lo) * 1.0001f;
        if (weight_call(z, c->ws) < c->least) return miss(kToMin);
    }
    return kDone;
}

// A slice's tokens that surely stay go into its batches' mass, those of the
// bins that may hold the end into the first CTA's `fine`.
template <int DT>
__device__ __noinline__ void keep_tokens(const Cluster& cl, const Smem& s, const Ctrl* c0, float z_hi, float per_bin,
                                         const WeightScale ws) {
    constexpr int BEL = kBatchVecs * Row<DT>::EPV;
    const int n = (int)min(s.c->count, (uint32_t)kBracketCap);
    const bool by_min = c0->by_min;
    const int f0 = c0->first_bin, f1 = c0->last_bin;
    const uint64_t least = s.c->least;
    uint64_t* end = cl.at(s.fine, 0);
    uint32_t* count = &cl.at(s.c, 0)->runs;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint64_t e = s.buf[i];
        const int bin = by_min ? 0 : fine_bin(e, z_hi, per_bin);
        if (by_min || bin < f0) {
            const uint64_t w = weight_call(candidate_value(e), ws);
            if (w >= least) shared_add(&s.bmass[(uint32_t)e / BEL], w);
        } else if (bin <= f1) {
            const uint32_t at = atomicAdd(count, 1u);
            if (at < (uint32_t)kFine) end[at] = e;
        }
    }
}

// The last step of a pass, in the first CTA: the tokens around the nucleus' end
// in order, the kept mass, and the token.  The last tier's token stands
// whatever its distance from a border.  Returns the next verdict.
template <int DT>
__device__ __noinline__ int end_row(const RowSearchArgs& a, const Smem& s, const char* row, int64_t V, int nb,
                                    int64_t o, int tier) {
    constexpr int BEL = kBatchVecs * Row<DT>::EPV;
    Ctrl* c = s.c;
    const int t = threadIdx.x;
    uint64_t slack = 0, sure = ~0ull;
    const uint64_t err = c->err;
    if (c->top_p < 1.f && !c->by_min) {
        const uint64_t before_bin = c->left, t_lo = c->t_lo, t_mid = c->t_mid, t_hi = c->t_hi;
        const int n = (int)c->runs;
        if (n > kFine) return kRadix;
        __syncthreads();
        auto crossing = [&](uint64_t e, uint64_t m0, uint64_t w) {
            const uint64_t next = m0 + w;
            if (m0 < t_lo && next >= t_lo) {
                c->sure = e;
                c->sure_mass = next;
            }
            if (m0 < t_mid && next >= t_mid) {
                c->cut_key = ~(uint32_t)(e >> 32);
                c->cut_last = (uint32_t)e;
                c->left = next;
            }
            if (m0 < t_hi && next >= t_hi) c->slack = next;
            if (m0 < t_mid) shared_add(&s.bmass[(uint32_t)e / BEL], w);
        };
        if (n <= kThreads) {
            const uint64_t mine = t < n ? s.fine[t] : ~0ull;
            const uint64_t w = t < n ? weight_call(candidate_value(mine), c->ws) : 0ull;
            if (t < n) s.buf[t] = w;
            __syncthreads();
            if (t < n) {
                uint64_t m0 = before_bin;
#pragma unroll 4
                for (int j = 0; j < n; ++j) m0 += s.fine[j] < mine ? s.buf[j] : 0ull;
                crossing(mine, m0, w);
            }
        } else {
            sort_u64(s.fine, n, s.buf, c);
            const int per = (n + kThreads - 1) / kThreads, i0 = min(n, t * per), i1 = min(n, i0 + per);
            uint64_t mine = 0, all;
            for (int i = i0; i < i1; ++i) mine += weight_call(candidate_value(s.fine[i]), c->ws);
            uint64_t m0 = before_bin + block_scan(mine, c->scan, all);
            for (int i = i0; i < i1; ++i) {
                const uint64_t w = weight_call(candidate_value(s.fine[i]), c->ws);
                crossing(s.fine[i], m0, w);
                m0 += w;
            }
        }
        if (t == 0) {
            c->cut_ties = 0xffffffffu;
            c->ties_before = 0;
        }
        __syncthreads();
        sure = c->sure;
        slack = max(c->slack - c->left, c->left - c->sure_mass);
    } else if (t == 0) {  // everything, or (the walk looks at the weights) what min-p keeps
        c->cut_key = kKeyNegInf;
        c->cut_ties = 0;
        c->cut_last = 0;
        c->ties_before = 0;
    }
    __syncthreads();
    find_batch(s, nb, 0, 0);
    // min-p ends the row only if its tokens are all inside the nucleus
    if (c->by_min && c->top_p < 1.f && add_up_to_most(c->mass, 2 * err) >= scale_ceil(c->total, c->top_p)) {
        __syncthreads();
        if (t == 0) {
            const float hi = c->z_hi, width = hi - c->z_lo;
            c->z_lo = hi - 1.1f * width;
            c->z_hi = hi + 4.f * width;
            c->by_min = 0;
            c->tries += 1;
        }
        __syncthreads();
        return c->tries < kTries ? tier : (int)kRadix;
    }
    const bool first = c->u == 0.f;
    if (!first) {
        walk_batch<DT>(row, V, c);
    } else {
        if (t < 32) {
            const int token = first_kept<DT>(row, V, nb, c);
            if (t == 0) {
                c->token = token;
                c->z = token >= 0 ? Row<DT>::scalar(row, token) : 0.f;
            }
        }
        __syncthreads();
    }
    // the token has to be further from its borders than the sums' error and
    // the slack of the kept mass, to stay whichever token ends the nucleus, and
    // prob to be within 2^-17
    const uint64_t off = slack + err / 2 + 1;
    bool done = c->token >= 0;
    if (done && tier != kTier3)
        done = slack <= (c->mass >> 17) && (first || well_inside(c->lo_side, c->left, c->hi_side, off)) &&
               candidate(c->z, (uint32_t)c->token) <= sure;
    if (t == 0 && done) write_token(a, c, o, c->token, c->z, c->mass);
    return done ? (int)kDone : tier == kTier3 ? (int)kRadix : tier + 1;
}

// The other slices' lists behind the first CTA's own (`count` of them may
// exceed `cap`, then the list is cut off).
__device__ __forceinline__ void join_lists(const Cluster& cl, const Smem& s, uint32_t cap) {
    uint32_t n = s.c->count;
    for (int rk = 1; rk < cl.split; ++rk) {
        const uint64_t* rb = cl.at(s.buf, rk);
        const uint32_t m = cl.at(s.c, rk)->count;
        for (uint32_t i = threadIdx.x; i < m && n + i < cap; i += kThreads) s.buf[n + i] = rb[i];
        n += m;
    }
    __syncthreads();
    if (threadIdx.x == 0) s.c->count = n;
    __syncthreads();
}

__device__ __forceinline__ void join_masses(const Cluster& cl, const Smem& s, int nb, int per) {
    for (int i = per + (int)threadIdx.x; i < nb; i += kThreads) s.bmass[i] = cl.at(s.bmass, i / per)[i];
    __syncthreads();
}

// The first cut_ties positions at cut_key, after the c->count candidates that
// buf holds (one warp).
template <int DT>
__device__ __noinline__ void first_ties(const char* row, int64_t V, int nb, uint32_t cut_key, uint32_t cut_ties,
                                        uint64_t* buf, Ctrl* c) {
    constexpr int EPV = Row<DT>::EPV;
    const int lane = threadIdx.x & 31;
    const uint32_t base = c->count;
    uint32_t found = 0;
    for (int v0 = 0; v0 < nb * kBatchVecs && found < cut_ties; v0 += 32) {
        float z[EPV];
        Row<DT>::unpack(load_vec<DT>(row, V, v0 + lane), z);
        uint32_t mine = 0;
#pragma unroll
        for (int e = 0; e < EPV; ++e) mine += key_of(z[e]) == cut_key;
        uint32_t inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(DLM_FULL_MASK, inc, o);
            if (lane >= o) inc += x;
        }
        uint32_t rank = found + inc - mine;
#pragma unroll
        for (int e = 0; e < EPV; ++e)
            if (key_of(z[e]) == cut_key) {
                if (rank < cut_ties && base + rank < (uint32_t)kCap)
                    buf[base + rank] = candidate(z[e], (uint32_t)((v0 + lane) * EPV + e));
                ++rank;
            }
        found += __shfl_sync(DLM_FULL_MASK, inc, 31);
    }
    __syncwarp();
    if (lane == 0) c->count = base + min(found, cut_ties);
}

// ---- the kernels -----------------------------------------------------------

__device__ void write_topk(const RowSearchArgs& a, const Smem& s, int n, int64_t o) {
    for (int i = threadIdx.x; i < a.k; i += kThreads) {
        a.values[o * a.k + i] = i < n ? candidate_value(s.buf[i]) : -INFINITY;
        a.ids[o * a.k + i] = i < n ? (int32_t)(uint32_t)s.buf[i] : -1;
    }
}

// The first CTA's decision after the first pass, from few candidates or from
// the batch sums.  Returns the verdict.
template <int DT>
__device__ __forceinline__ int sample_leader(const RowSearchArgs& a, const Smem& s, const char* row, int64_t V, int nb,
                                             int64_t o, bool whole, float low) {
    Ctrl* c = s.c;
    const int t = threadIdx.x, nsub = nb * kRuns;
    const int k = c->top_k;
    const float p = c->top_p, m = c->ws.m;
    const bool by_p = p < 1.f, by_least = c->least > 0;
    const float z_least = by_least ? min_p_logit(c) : -INFINITY;
    ListRule rule{k > 0 ? k : 0x7fffffff, true, true};
    float least;
    if (whole) {
        least = -INFINITY;
    } else if (k > 0) {
        // (more than the runs: a list from a threshold that a sample gives)
        least = k == 1 ? m : k <= DLM_MAX_TOPK ? threshold_for(s.sub, nsub, k, low, m, c) : -INFINITY;
        if (!(least > -INFINITY)) return k <= kListTopk ? kList : kRadix;
    } else if (by_least) {
        least = z_least;
        rule.complete = !by_p;
    } else if (by_p) {
        rule.complete = rule.all_least = false;
        uint64_t lo, hi;
        nucleus_target(c, rule, 0, lo, hi);
        least = m;
        if (hi > kOne) {  // more than the largest logit alone
            least = threshold_for(s.sub, nsub, min(kListRuns, nb), low, m, c);
            // what the runs' maxima hold of the nucleus: a list of the runs
            // that is far short of it is not made
            float v = 0.f;
            if (least > -INFINITY)
                for (int i = t; i < nsub; i += kThreads)
                    if (s.sub[i] >= least) v += ex2((s.sub[i] - m) * c->ws.c_hi);
            uint64_t held;
            block_scan((uint64_t)__float2ull_rn(v * 17592186044416.0f), c->scan, held);
            if (held + held / 2 < hi) return kTier1;
        }
    } else {
        // no filter: the batch sums lead to the token, if it is further than
        // their error from a border
        if (c->u == 0.f) return kTier1;
        if (t == 0) {
            c->cut_key = kKeyNegInf;
            c->cut_ties = c->cut_last = c->ties_before = 0;
        }
        find_batch(s, nb, 0, 0);
        walk_batch<DT>(row, V, c);
        // every weight off by a share e at most, a running sum of the share u
        // of the mass and u times the whole differ by at most 2 u (1 - u) e of
        // the mass from what they should: e / 2
        const uint64_t off = c->margin / 2 + 1;
        const bool sure = c->token >= 0 && well_inside(c->lo_side, c->left, c->hi_side, off);
        if (t == 0 && sure) write_token(a, c, o, c->token, c->z, c->mass);
        return sure ? kDone : kTier1;
    }
    gather_runs<DT>(row, V, nsub, s, least);
    // a top-k's ties go over the whole row
    const int other = k == 0 ? kTier1 : kRadix;
    if (c->count > (uint32_t)kCap) return other;
    const uint32_t n = k > 0 ? (uint32_t)top_candidates(s, (int)c->count, k) : c->count;
    if (n <= (uint32_t)kThreads) return decide_small(a, s, (int)n, rule, o) ? kDone : other;
    sort_u64(s.buf, (int)n, s.wbuf, c);
    keep_candidates(s, (int)n, rule);
    const int kept = c->n;
    if (kept <= 0) return other;
    pick_candidate<DT>(a, s, kept, row, o);
    return kDone;
}

// A row's settings into ctrl (one thread of each CTA of its cluster).
template <bool SAMPLE>
__device__ __forceinline__ void load_settings(const RowSearchArgs& a, int64_t o, Ctrl* c, const uint64_t* tab) {
    float T = a.temperature, p = a.top_p, least = a.min_p;
    int k = a.k;
    bool bad = false;
    if constexpr (SAMPLE) {
        if (a.temperature_rows) T = a.temperature_rows[o];
        if (a.top_k_rows) k = a.top_k_rows[o];
        if (a.top_p_rows) p = a.top_p_rows[o];
        if (a.min_p_rows) least = a.min_p_rows[o];
        const float u = a.uniform[o];
        bad = !(T == 0.f || (T >= DLM_MIN_TEMPERATURE && T <= DLM_MAX_TEMPERATURE)) || k < 0 || !(p > 0.f && p <= 1.f) ||
              !(least >= 0.f && least <= 1.f) || !(u >= 0.f && u < 1.f);
        c->u = u;
        if (T == 0.f) k = 1, T = 1.f, p = 1.f, least = 0.f;  // the argmax
        if (k >= a.vocab) k = 0;
    }
    c->bad = bad;
    c->top_k = k;
    c->top_p = p;
    c->min_p = least;
    c->least = bad ? 0 : least < 1.f ? scale_ceil(kOne, least) : kOne;
    c->ws = weight_scale(0.f, bad ? 1.f : T);
    c->ws.tab = tab;
}

__device__ __forceinline__ void write_none(const RowSearchArgs& a, int64_t o) {
    a.token[o] = -1;
    a.prob[o] = 0.f;
    if (a.conf) a.conf[o] = 0.f;
}

// A CTA's share of a row.
struct Work {
    const char* row;
    int64_t o;    // where the row's results go
    int nb, per, b0, b1;
    __device__ Work(const RowSearchArgs& a, const Cluster& cl, int64_t q, int64_t out, int esz, int bel) {
        row = static_cast<const char*>(a.logits) + q * a.row_stride * esz;
        o = out;
        nb = (int)((a.vocab + bel - 1) / bel);
        per = (nb + cl.split - 1) / cl.split;
        b0 = min(nb, cl.rank * per);
        b1 = min(nb, b0 + per);
    }
};

// What the first pass left open, by every CTA of the row's cluster: the tiers
// from `verdict` on, then the radix search.  Ctrl holds the row's settings in
// every CTA, and in the first one the maximum and the bracket.
template <int DT, bool SAMPLE>
__device__ __forceinline__ void finish_row(const RowSearchArgs& a, const Cluster& cl, const Smem& s, const Work& w,
                                           int verdict) {
    const int t = threadIdx.x, nb = w.nb;
    const int64_t V = a.vocab, o = w.o;
    const char* row = w.row;
    Ctrl* c = s.c;
    const Ctrl* c0 = cl.at(c, 0);
    WeightScale ws = c0->ws;
    ws.tab = s.tab;  // (this CTA's)
    if constexpr (SAMPLE) {
        while (verdict >= kTier1 && verdict <= kTier3) {
            const float z_lo = c0->z_lo, z_hi = c0->z_hi, per_bin = (float)kFine / (z_hi - z_lo);
            const bool bins = c->top_p < 1.f && !c0->by_min;
            if (t == 0) c->count = 0;
            __syncthreads();
            float* fine = reinterpret_cast<float*>(s.fine);
            if (verdict == kTier1)
                bracket_pass<DT, 1>(row, V, w.b0, w.b1, z_lo, z_hi, ws, s.bmass, c, s.buf, fine);
            else if (verdict == kTier2)
                bracket_pass<DT, 2>(row, V, w.b0, w.b1, z_lo, z_hi, ws, s.bmass, c, s.buf, fine);
            else
                bracket_pass<DT, 3>(row, V, w.b0, w.b1, z_lo, z_hi, ws, s.bmass, c, s.buf, fine);
            if (bins) bin_tokens(s, z_hi, per_bin, ws);
            cl.sync();
            if (bins && cl.split > 1) {
                merge_bins(cl, s.fine, kFine);
                cl.sync();
            }
            if (cl.rank == 0) {
                const int next = find_end(cl, s, nb, verdict);
                if (t == 0) c->verdict = next;
            }
            cl.sync();
            if (c0->verdict == kDone) {  // the end is inside the bracket
                keep_tokens<DT>(cl, s, c0, z_hi, per_bin, ws);
                cl.sync();
                if (cl.rank == 0) {
                    join_masses(cl, s, nb, w.per);
                    const int next = end_row<DT>(a, s, row, V, nb, o, verdict);
                    __syncthreads();
                    if (t == 0) c->verdict = next;
                }
                cl.sync();
            }
            verdict = c0->verdict;
            cl.sync();  // (read before the first CTA sets it again)
        }
        if (verdict == kDone) return;
    }
    if (verdict == kList) {
        if (t == 0) c->count = 0;
        __syncthreads();
        gather_slice<DT>(row, V, w.b0, w.b1, c0->z_lo, s.buf, &c->count);
        cl.sync();
        if (cl.rank == 0) {
            join_lists(cl, s, kCap);
            const int n = (int)c->count, k = c->top_k;
            const bool fits = n >= k && n <= kCap;
            if (fits) {
                sort_u64(s.buf, n, s.wbuf, c);
                if constexpr (!SAMPLE) {
                    write_topk(a, s, k, o);
                } else {
                    keep_candidates(s, n, ListRule{k, true, true});
                    pick_candidate<DT>(a, s, c->n, row, o);
                }
            }
            if (t == 0) c->verdict = fits ? kDone : kRadix;
        }
        cl.sync();
        verdict = c0->verdict;
        cl.sync();
        if (verdict == kDone) return;
    }
    cl.sync();

    // the search over the whole row
    const int k = c->top_k;
    uint32_t cut_key = kKeyNegInf, cut_ties = 0;
    if (k > 0) {
        bool list;
        count_cut<DT>(cl, s, row, V, w.b0, w.b1, k, ws, cut_key, cut_ties, list);
        if (!SAMPLE || list) {
            // the list, once more: every key from the cut on (or, when the
            // last key's ties overflow it, the keys above and the first ties)
            if (t == 0) c->count = 0;
            __syncthreads();
            gather_slice<DT>(row, V, w.b0, w.b1, key_value(list ? cut_key : cut_key + 1), s.buf, &c->count);
            cl.sync();
            if (cl.rank == 0) {
                join_lists(cl, s, kCap);
                if (!list) {
                    if (t < 32) first_ties<DT>(row, V, nb, cut_key, cut_ties, s.buf, c);
                    __syncthreads();
                }
                const int n = (int)c->count;
                sort_u64(s.buf, n, s.wbuf, c);
                if constexpr (!SAMPLE) {
                    write_topk(a, s, min(n, k), o);
                } else {
                    keep_candidates(s, n, ListRule{k, true, true});
                    pick_candidate<DT>(a, s, c->n, row, o);
                }
            }
            cl.sync();
            return;
        }
    }
    if constexpr (SAMPLE) {
        if (c->top_p < 1.f) {
            uint32_t key, ties;
            mass_cut<DT>(cl, s, row, V, w.b0, w.b1, c->top_p, cut_key, cut_ties, ws, key, ties);
            cut_key = key;
            cut_ties = ties;
        }
        batch_masses<DT>(row, V, w.b0, w.b1, cut_key, c->least, ws, s.bmass, s.bties);
        cl.sync();
        if (cl.rank == 0) {
            join_masses(cl, s, nb, w.per);
            for (int i = w.per + t; i < nb; i += kThreads) s.bties[i] = cl.at(s.bties, i / w.per)[i];
            if (t == 0) {
                c->cut_key = cut_key;
                c->cut_ties = cut_ties;
                c->cut_last = 0xffffffffu;
                c->ties_before = 0;
            }
            __syncthreads();
            uint64_t w_tie = cut_key > kKeyNegInf && cut_ties > 0 ? weight_call(key_value(cut_key), ws) : 0;
            if (w_tie < c->least) w_tie = 0;
            find_batch(s, nb, w_tie, cut_ties);
            if (c->u > 0.f) {
                walk_batch<DT>(row, V, c);
                if (t == 0) write_token(a, c, o, max(c->token, 0), c->z, c->mass);
            } else if (t < 32) {
                const int token = max(first_kept<DT>(row, V, nb, c), 0);
                if (t == 0) write_token(a, c, o, token, Row<DT>::scalar(row, token), c->mass);
            }
        }
        cl.sync();
    }
}

// A row that the first launch leaves to the second: bits 24..26 of its token
// hold the verdict, below them the bracket's bins; the sign marks it (a token
// of -1, a row without one, has the bits above 26 set).  Its maximum is in prob.
constexpr uint32_t kOpenMask = 0xf8000000u, kOpenMark = 0x80000000u, kClaimed = 0x08000000u;

// DEFER: rows that the first pass leaves open go to open_rows_kernel.
template <int DT, bool SAMPLE, bool DEFER>
__global__ void __launch_bounds__(kThreads, 4) row_search_kernel(const RowSearchArgs a) {
    extern __shared__ __align__(16) unsigned char s_raw[];
    const int t = threadIdx.x;
    if (DEFER) asm volatile("griddepcontrol.launch_dependents;");
    Cluster cl;
    cl.split = DEFER ? 1 : a.split;
    const int64_t r = blockIdx.x / cl.split;
    cl.rank = (int)(blockIdx.x - r * cl.split);
    const int64_t q = a.row_index ? (int64_t)a.row_index[r] : r;
    if (q < 0 || (a.n_src > 0 && q >= a.n_src)) {  // the same for every CTA of the cluster
        if (cl.rank == 0 && t == 0) raise_status(a.dev_status, DLM_DEV_BAD_INDEX);
        return;
    }
    const int64_t V = a.vocab;
    const Work w(a, cl, q, a.gather ? r : q, Row<DT>::ESZ, kBatchVecs * Row<DT>::EPV);
    const int nb = w.nb;
    const int64_t o = w.o;
    const Smem s = carve(s_raw, nb);
    Ctrl* c = s.c;

    // Every logit of a short row fits the list, if a filter makes one.  A
    // top-k within the list needs no sums, and min-p without top-p neither.
    bool filtered = true, whole = false, sums = true;
    c->bins[t] = 0;
    static_assert(kThreads == 256, "one entry of the table per thread");
    s.tab[t] = kPow2Neg[t];
    float low = INFINITY;
    // the maxima and sums go straight to the first CTA, which has to run by then
    if (cl.split > 1) cg::this_cluster().barrier_arrive();
    const float most = scan_rows<DT>(w.row, V, w.b0, w.b1, [&]() {
        if (t == 0) load_settings<SAMPLE>(a, o, c, s.tab);
        __syncthreads();
        if (SAMPLE && c->bad) return -1.f;
        filtered = c->top_k > 0 || c->top_p < 1.f || c->least > 0;
        whole = V <= kCap && filtered;
        sums = !SAMPLE || (c->top_k == 0 && !whole && (c->top_p < 1.f || c->least == 0));
        if (cl.split > 1) cg::this_cluster().barrier_wait();
        return sums ? c->ws.c_hi : 0.f;
    }, cl.at(s.sub, 0), cl.at(s.bsum, 0), low);
    if (SAMPLE && c->bad) {
        if (cl.split > 1) cg::this_cluster().barrier_wait();
        if (cl.rank == 0 && t == 0) {
            write_none(a, o);
            raise_status(a.dev_status, DLM_DEV_BAD_PARAM);
        }
        return;
    }
    const int k = c->top_k;
    if ((t & 31) == 0) {
        cl.at(c, 0)->wmax[cl.rank * kWarps + (t >> 5)] = most;
        cl.at(c, 0)->wmin[cl.rank * kWarps + (t >> 5)] = low;
    }
    cl.sync();

    int found = kDone;
    if (cl.rank == 0) {
        float m = -INFINITY;
        low = INFINITY;
        for (int i = t & 31; i < cl.split * kWarps; i += 32) {  // every warp for itself
            m = max_nan(m, c->wmax[i]);
            low = fminf(low, c->wmin[i]);
        }
        m = warp_max_nan(m);
        low = -warp_max_nan(-low);
        if (t == 0) c->ws.m = m;
        __syncthreads();
        int verdict = kDone;
        if (!(m > -INFINITY && m < INFINITY)) {  // NaN, +inf, or nothing but -inf
            if constexpr (SAMPLE) {
                if (t == 0) write_none(a, o);
            } else {
                write_topk(a, s, 0, o);
                if (t == 0 && a.lse) a.lse[o] = m;  // -inf, +inf or NaN
            }
            if (t == 0) raise_status(a.dev_status, DLM_DEV_NONFINITE);
        } else {
            if (sums) {
                const WeightScale ws = c->ws;
                uint64_t v = 0, total;
                for (int b = t; b < nb; b += kThreads) {
                    const uint64_t x = batch_mass(s.sub, s.bsum, b, ws);
                    s.bmass[b] = x;
                    v += x;
                }
                block_scan(v, c->scan, total);
                // the sums' error, in 2^-24: 4 for each ex2 (the weight's and
                // its batch's), 12 for eleven levels of additions and the
                // products, 2.1 per unit of exponent (three roundings), whose
                // mean over the mass is at most log2 V less log2 of the mass
                if (t == 0) {
                    c->total = total;
                    const float mean = fmaxf(0.f, __log2f((float)V) + 0.01f - __log2f((float)total * 0x1p-44f));
                    c->margin = (total >> 24) * (uint64_t)(21.f + 2.1f * mean) + nb;
                    if (!SAMPLE && a.lse) a.lse[o] = m / a.temperature + logf((float)total * 0x1p-44f);
                }
                __syncthreads();
            }
            if constexpr (SAMPLE) {
                verdict = sample_leader<DT>(a, s, w.row, V, nb, o, whole, low);
                // logits so far from 0 that tiers 1 and 2 can not tell "60 powers
                // of 2 below the maximum" from the maximum itself
                if (verdict == kTier1 && fabsf(m) * c->ws.c_hi > 60.f * 1048576.f) verdict = kRadix;
            } else {
                const float least = whole ? -INFINITY : threshold_for(s.sub, nb * kRuns, k, low, m, c);
                verdict = kRadix;
                if (!whole && !(least > -INFINITY)) {
                    verdict = kList;
                } else {
                    gather_runs<DT>(w.row, V, nb * kRuns, s, least);
                    if (c->count <= (uint32_t)kCap) {
                        const int n = top_candidates(s, (int)c->count, k);
                        sort_u64(s.buf, n, s.wbuf, c);
                        write_topk(a, s, min(n, k), o);
                        verdict = kDone;
                    }
                }
            }
        }
        found = verdict;
        if (t == 0) c->verdict = verdict;
    }
    // a row that needs a bracket or a list's threshold: a sample of it by all its CTAs
    if (!DEFER) {
        cl.sync();
        found = cl.at(c, 0)->verdict;
        if (found == kDone) {
            cl.sync();  // (the first CTA's ctrl has been read)
            return;
        }
    }
    int verdict = found;
    if (verdict == kList || (verdict == kTier1 && filtered)) {
        float scale = 1.f;
        if (verdict == kList || c->top_p < 1.f) {
            // half the sample is enough for the largest k of dlm_row_topk (48 and 44 us
            // for the 1000 largest of 61 rows of 100003 floats)
            const int tokens = verdict == kList && k <= DLM_MAX_TOPK ? kSampleTokens / 2 : kSampleTokens;
            scale = sample_row<DT>(cl, w.row, V, s, tokens, cl.at(c, 0)->ws.m, c->ws.c_hi);
            if (cl.split > 1) {
                cl.sync();
                merge_bins(cl, reinterpret_cast<uint32_t*>(s.buf), kBins);
                cl.sync();
            }
        }
        if (cl.rank == 0) verdict = verdict == kList ? place_list(k, s, scale) : place_bracket(s, scale);
    }
    if (DEFER) {
        if (t == 0 && verdict != kDone) {
            const bool placed = verdict == kMinP || verdict == kList || (verdict == kTier1 && filtered);
            const uint32_t bins = placed ? (uint32_t)c->bin_lo << 12 | (uint32_t)(verdict == kList ? 0 : c->bin_hi) : 0u;
            a.token[o] = (int32_t)(kOpenMark | (uint32_t)verdict << 24 | bins);
            a.prob[o] = c->ws.m;
        }
        return;
    }
    if (cl.rank == 0 && t == 0) {
        set_bracket(c, verdict);
        c->verdict = verdict == kMinP ? kTier1 : verdict;
    }
    cl.sync();
    finish_row<DT, SAMPLE>(a, cl, s, w, cl.at(c, 0)->verdict);
}

// The rows that row_search_kernel left open.  Which rows they are is not known
// at the launch, and a cluster takes tens of microseconds for one, so clusters
// claim them: the first CTA looks for a marked token, each cluster from its own
// place in the batch on, and changes the mark to a claimed one.  (Rows i,
// i + clusters, ... for cluster i, without claims: the cluster with the most
// open rows had twice the average and set the time, 440 us for 839 rows.)
template <int DT>
__global__ void __launch_bounds__(kThreads, 4) open_rows_kernel(const RowSearchArgs a) {
    extern __shared__ __align__(16) unsigned char s_raw[];
    __shared__ unsigned long long s_pick;
    __shared__ int64_t s_row;
    __shared__ uint32_t s_mark;
    const int t = threadIdx.x;
    Cluster cl;
    cl.split = a.split;
    cl.rank = (int)(blockIdx.x % a.split);
    const int64_t place = (int64_t)(blockIdx.x / a.split) * a.n_rows / (gridDim.x / a.split);
    constexpr int BEL = kBatchVecs * Row<DT>::EPV;
    const Smem s = carve(s_raw, (int)((a.vocab + BEL - 1) / BEL));
    Ctrl* c = s.c;
    s.tab[t] = kPow2Neg[t];
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the first launch's marks
    int64_t from = 0;  // rows looked at, from `place` on, that are not open any more
    while (true) {
        if (cl.rank == 0) {
            if (t == 0) s_row = -1;
            while (from < a.n_rows) {
                // the first marked row of the next kThreads
                if (t == 0) s_pick = ~0ull;
                __syncthreads();
                const int64_t i = from + t;
                int64_t r = place + i;
                if (r >= a.n_rows) r -= a.n_rows;
                const int64_t q = i >= a.n_rows ? -1 : a.row_index ? (int64_t)a.row_index[r] : r;
                if (q >= 0 && !(a.n_src > 0 && q >= a.n_src)) {
                    const int32_t mark = *(const volatile int32_t*)(a.token + (a.gather ? r : q));
                    if (((uint32_t)mark & kOpenMask) == kOpenMark) atomicMin(&s_pick, (unsigned long long)i);
                }
                __syncthreads();
                const unsigned long long pick = s_pick;
                __syncthreads();
                if (pick == ~0ull) {
                    from += kThreads;
                    continue;
                }
                if (t == 0) {
                    int64_t row = place + (int64_t)pick;
                    if (row >= a.n_rows) row -= a.n_rows;
                    const int64_t o = a.gather || !a.row_index ? row : (int64_t)a.row_index[row];
                    const int32_t mark = *(const volatile int32_t*)(a.token + o);
                    if (((uint32_t)mark & kOpenMask) == kOpenMark &&
                        atomicCAS(a.token + o, mark, (int32_t)((uint32_t)mark | kClaimed)) == mark) {
                        s_row = row;
                        s_mark = (uint32_t)mark;
                    }
                }
                __syncthreads();
                from = (int64_t)pick + 1;
                if (s_row >= 0) break;
            }
        }
        cl.sync();
        const int64_t r = *cl.at(&s_row, 0);
        const uint32_t mark = *cl.at(&s_mark, 0);
        if (r < 0) break;
        const int64_t q = a.row_index ? (int64_t)a.row_index[r] : r;
        const Work w(a, cl, q, a.gather ? r : q, Row<DT>::ESZ, BEL);
        const int verdict = (int)(mark >> 24) & 7;
        if (t == 0) {  // every CTA of the cluster keeps the row's settings
            load_settings<true>(a, w.o, c, s.tab);
            c->ws.m = *(const volatile float*)(a.prob + w.o);
            c->bin_lo = (int)(mark >> 12) & 0xfff;
            c->bin_hi = (int)mark & 0xfff;
            set_bracket(c, verdict);
        }
        cl.sync();
        finish_row<DT, true>(a, cl, s, w, verdict == kMinP ? kTier1 : verdict);
    }
    cl.sync();  // (the first CTA's choice has been read)
}

template <int DT>
size_t smem_for(int64_t V, bool fine) {
    constexpr int BEL = kBatchVecs * Row<DT>::EPV;
    return smem_bytes((int)((V + BEL - 1) / BEL), fine);
}

template <int DT, typename F>
cudaError_t launch_rows(F kernel, const RowSearchArgs& a, int64_t grid, bool fine, bool programmatic, cudaStream_t st) {
    const size_t smem = smem_for<DT>(a.vocab, fine);
    if (smem > 47 * 1024) {  // (static shared memory on top) the same limit whatever the call's size: calls may run side by side
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)smem_for<DT>(DLM_MAX_SEARCH_VOCAB, true));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (a.split > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = a.split;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (programmatic) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = n ? attr : nullptr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int DT>
cudaError_t launch_sample(const RowSearchArgs& a, cudaStream_t st) {
    // rows of fewer batches than two per warp are finished where they are: a
    // pass over one takes its CTA less than a launch does
    if (a.split > 1 || a.vocab <= 2 * kWarps * kBatchVecs * Row<DT>::EPV)
        return launch_rows<DT>(row_search_kernel<DT, true, false>, a, a.n_rows * a.split, true, false, st);
    const cudaError_t e = launch_rows<DT>(row_search_kernel<DT, true, true>, a, a.n_rows, false, false, st);
    if (e != cudaSuccess) return e;
    RowSearchArgs open = a;
    open.split = kOpenSplit;
    const int64_t slots = (int64_t)a.num_sms * 4 / kOpenSplit, clusters = a.n_rows < slots ? a.n_rows : slots;
    return launch_rows<DT>(open_rows_kernel<DT>, open, clusters * kOpenSplit, true, true, st);
}

template <int DT>
cudaError_t launch_topk(const RowSearchArgs& a, cudaStream_t st) {
    return launch_rows<DT>(row_search_kernel<DT, false, false>, a, a.n_rows * a.split, false, false, st);
}

}  // namespace

// CTAs per row: a row is split over a cluster when the rows alone do not fill
// the GPU and every warp still gets a batch.
int row_search_split(int dtype, int64_t n_rows, int64_t vocab, int num_sms) {
    const int64_t nb = vocab / (kBatchVecs * (dtype == DLM_F32 ? 4 : 8));
    int split = 1;
    while (split < 8 && n_rows * split < 2LL * num_sms && nb / (split * 2) >= kWarps) split *= 2;
    return split;
}

cudaError_t launch_row_topk(const RowSearchArgs& a, int dtype, cudaStream_t st) {
    switch (dtype) {
    case DLM_BF16: return launch_topk<DLM_BF16>(a, st);
    case DLM_F16: return launch_topk<DLM_F16>(a, st);
    default: return launch_topk<DLM_F32>(a, st);
    }
}

cudaError_t launch_row_sample(const RowSearchArgs& a, int dtype, cudaStream_t st) {
    switch (dtype) {
    case DLM_BF16: return launch_sample<DLM_BF16>(a, st);
    case DLM_F16: return launch_sample<DLM_F16>(a, st);
    default: return launch_sample<DLM_F32>(a, st);
    }
}

}  // namespace dlm
