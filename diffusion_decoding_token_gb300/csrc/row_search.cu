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
// candidates are sorted and decided with 64-bit integer weights (weight.cuh).
// A row whose filters keep more than the candidate list holds is searched
// over the whole row: radix passes over the ordered keys with counts (top-k)
// or 64-bit masses (top-p), then one pass for the kept mass of each batch.
//
// A row is worked by one CTA, or by a cluster of CTAs when rows are few.
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
constexpr int kBins = 2048;            // radix bins of a pass over the whole row
constexpr uint32_t kKeyNegInf = 0x007fffffu;  // ordered key of -inf
static_assert(kCap >= 2 * DLM_MAX_TOPK, "a candidate list holds the largest top-k and ties");

// Keys whose unsigned order is the order of the floats; -0 counts as +0.
__device__ __forceinline__ uint32_t key_of(float z) {
    const uint32_t b = __float_as_uint(z + 0.0f);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// What one row's CTA (the first of its cluster) and the others share.
struct Ctrl {
    WeightScale ws;
    float temperature, top_p, u;
    float z_least;        // min-p: the smallest logit that stays
    int top_k;            // 0: off
    int bad;              // a parameter of this row is out of range
    int done;             // the row's outputs are written
    uint32_t count;       // candidates found (may exceed kCap)
    int n;                // tokens kept, or -1
    // the search over the whole row
    uint32_t prefix;      // key bits found so far
    uint64_t above;       // count or mass of the keys above the prefix
    uint64_t total;
    uint32_t cut_key;     // kept: keys above cut_key, and the first cut_ties positions at it
    uint32_t cut_ties;
    uint64_t scan[kWarps];
    float fscan[kWarps];
    uint64_t mass;        // kept mass
    uint64_t left;        // target inside the chosen batch
    int batch;
    uint32_t ties_before;
    uint64_t margin;
};

// Shared memory of a CTA: sub[4 nb] run maxima, bsum[nb] batch sums, bmass[nb]
// and bties[nb] of the whole-row search, buf[kCap] candidates (or radix bins)
// and wbuf[kCap] their weights.
struct Smem {
    Ctrl* c;
    uint64_t* buf;
    uint64_t* wbuf;
    uint64_t* bmass;
    uint32_t* bties;
    float* sub;
    float* bsum;
};

__host__ __device__ inline size_t ctrl_bytes() { return (sizeof(Ctrl) + 15) & ~(size_t)15; }

__device__ __forceinline__ Smem carve(unsigned char* p, int nb) {
    Smem s;
    s.c = reinterpret_cast<Ctrl*>(p);
    p += ctrl_bytes();
    s.buf = reinterpret_cast<uint64_t*>(p);
    p += sizeof(uint64_t) * kCap;
    s.wbuf = reinterpret_cast<uint64_t*>(p);
    p += sizeof(uint64_t) * kCap;
    s.sub = reinterpret_cast<float*>(p);  // 16-byte aligned: a batch's four maxima are stored at once
    p += sizeof(float) * nb * kRuns;
    s.bmass = reinterpret_cast<uint64_t*>(p);
    p += sizeof(uint64_t) * nb;
    s.bsum = reinterpret_cast<float*>(p);
    p += sizeof(float) * nb;
    s.bties = reinterpret_cast<uint32_t*>(p);
    return s;
}

size_t smem_bytes(int nb) {
    return ctrl_bytes() + sizeof(uint64_t) * (2 * kCap + nb) + sizeof(float) * (size_t)nb * (kRuns + 2);
}

// Sort buf[0, n) ascending (n <= kCap).  Short lists by rank (every thread
// counts the smaller ones, broadcast reads, two barriers), longer ones by a
// bitonic network padded to a power of two.
__device__ void sort_u64(uint64_t* buf, int n) {
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
    int m = 512;
    while (m < n) m <<= 1;
    for (int i = n + threadIdx.x; i < m; i += kThreads) buf[i] = ~0ull;
    __syncthreads();
    for (int k = 2; k <= m; k <<= 1) {
        for (int j = k >> 1; j > 0; j >>= 1) {
            for (int i = threadIdx.x; i < m / 2; i += kThreads) {
                const int lo = 2 * i - (i & (j - 1)), hi = lo + j;
                const uint64_t a = buf[lo], b = buf[hi];
                if ((a > b) == ((lo & k) == 0)) {
                    buf[lo] = b;
                    buf[hi] = a;
                }
            }
            __syncthreads();
        }
    }
}

// A candidate: sorts by logit descending, then position ascending.
__device__ __forceinline__ uint64_t candidate(float z, uint32_t i) { return ((uint64_t)(~key_of(z)) << 32) | i; }
__device__ __forceinline__ float candidate_value(uint64_t c) { return key_value(~(uint32_t)(c >> 32)); }

// The k-th largest of the n floats of `sub` (-inf when n < k), by 8-bit radix
// passes over their keys; bins is kThreads words of scratch.
__device__ float kth_largest(const float* sub, int n, int k, uint32_t* bins, Ctrl* c) {
    if (n < k) return -INFINITY;
    uint32_t prefix = 0, left = (uint32_t)k;
    const int t = threadIdx.x;
    for (int shift = 24; shift >= 0; shift -= 8) {
        bins[t] = 0;
        __syncthreads();
        for (int i = t; i < n; i += kThreads) {
            const uint32_t key = key_of(sub[i]);
            if (shift == 24 || (key >> (shift + 8)) == prefix) atomicAdd(&bins[(key >> shift) & 255u], 1u);
        }
        __syncthreads();
        // thread t looks at bin 255 - t: the counts above it come from the scan
        uint64_t total;
        const uint32_t mine = bins[255 - t];
        const uint64_t before = block_scan(mine, c->scan, total);
        if (before < left && before + mine >= left) {
            c->prefix = (prefix << 8) | (uint32_t)(255 - t);
            c->above = before;
        }
        __syncthreads();
        prefix = c->prefix;
        left -= (uint32_t)c->above;
        __syncthreads();
    }
    return key_value(prefix);
}

// Push the elements z >= least of batches [b0, b1) into the list dst, its
// length in *count (both may be another CTA's of the cluster).  With `sub`,
// runs whose maximum is below `least` are skipped unread.
template <int DT>
__device__ void gather(const char* row, int64_t V, int b0, int b1, const float* sub, float least, uint64_t* dst,
                       uint32_t* count) {
    constexpr int EPV = Row<DT>::EPV;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int s = b0 * kRuns + warp; s < b1 * kRuns; s += kWarps) {
        if (sub && !(sub[s] >= least)) continue;
        const int v = s * 32 + lane;
        float z[EPV];
        Row<DT>::unpack(load_vec<DT>(row, V, v), z);
        int mine = 0;
#pragma unroll
        for (int e = 0; e < EPV; ++e) mine += z[e] >= least && z[e] > -INFINITY;
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(DLM_FULL_MASK, inc, o);
            if (lane >= o) inc += x;
        }
        uint32_t base = 0;
        const int all = __shfl_sync(DLM_FULL_MASK, inc, 31);
        if (all == 0) continue;
        if (lane == 0) base = atomicAdd(count, (uint32_t)all);
        base = __shfl_sync(DLM_FULL_MASK, base, 0) + (uint32_t)(inc - mine);
        if (mine) {
#pragma unroll
            for (int e = 0; e < EPV; ++e)
                if (z[e] >= least && z[e] > -INFINITY) {
                    if (base < (uint32_t)kCap) dst[base] = candidate(z[e], (uint32_t)(v * EPV + e));
                    ++base;
                }
        }
    }
}

// ---- the first pass --------------------------------------------------------

// Run maxima of batches [b0, b1), and with `sums` each batch's sum of
// 2^((z - ref) c), ref the batch's maximum (a batch of -inf only sums to 0).
template <int DT>
__device__ __forceinline__ void scan_rows(const char* row, int64_t V, int b0, int b1, bool sums, float c, float* sub,
                                          float* bsum) {
    constexpr int EPV = Row<DT>::EPV;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int b = b0 + warp; b < b1; b += kWarps) {
        uint4 w[kRuns];
        const int v0 = b * kBatchVecs + lane;
        if ((int64_t)(b + 1) * kBatchVecs * EPV <= V) {
#pragma unroll
            for (int i = 0; i < kRuns; ++i) w[i] = ld_stream(reinterpret_cast<const uint4*>(row) + v0 + i * 32);
        } else {
#pragma unroll
            for (int i = 0; i < kRuns; ++i) w[i] = load_vec<DT>(row, V, v0 + i * 32);
        }
        float m[kRuns];
#pragma unroll
        for (int i = 0; i < kRuns; ++i) m[i] = warp_max_nan(Row<DT>::vmax(w[i]));
        if (lane == 0) *reinterpret_cast<float4*>(sub + b * kRuns) = make_float4(m[0], m[1], m[2], m[3]);
        if (!sums) continue;
        const float ref = max_nan(max_nan(m[0], m[1]), max_nan(m[2], m[3]));
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
}

// A batch's sum relative to the row's maximum, in units of 2^-44.
__device__ __forceinline__ uint64_t batch_mass(const float* sub, const float* bsum, int b, const WeightScale& ws) {
    const float ref = fmaxf(fmaxf(sub[4 * b], sub[4 * b + 1]), fmaxf(sub[4 * b + 2], sub[4 * b + 3]));
    const float s = bsum[b] * ex2((ref - ws.m) * ws.c_hi);
    return ref > -INFINITY ? (uint64_t)__float2ull_rn(s * 17592186044416.0f) : 0ull;
}

// ---- candidates ------------------------------------------------------------

// Writes the row's token (thread-wise: the one thread that found it).
template <int DT>
__device__ __forceinline__ void write_token(const RowSearchArgs& a, const Ctrl* c, const char* row, int64_t o,
                                            int token, uint64_t mass) {
    const float z = Row<DT>::scalar(row, token);
    float lo;
    const float y = weight_exponent(z, c->ws, lo);
    // 2^-(y + lo) over the kept mass
    const float w = exp2f(-y) * fmaf(lo, -kLn2, 1.0f);
    a.token[o] = token;
    a.prob[o] = y < INFINITY ? fminf(1.0f, w / ((float)mass * 5.684341886080802e-14f)) : 0.f;
    if (a.conf) a.conf[o] = expf(z - a.lse_in[o]);
}

// How many of the N sorted candidates stay, and their mass.  K: candidates
// under the top-k (N when it is off).  `complete`: the list holds every token
// that any filter could keep; otherwise the row's mass is known only as
// total +- margin, the list holds its N largest tokens, and the result is -1
// when that does not decide.
__device__ void keep_candidates(const Smem& s, int K, bool complete) {
    Ctrl* c = s.c;
    const int t = threadIdx.x;
    const int per = (K + kThreads - 1) / kThreads, i0 = min(K, t * per), i1 = min(K, i0 + per);
    uint64_t sum = 0;
    for (int i = i0; i < i1; ++i) {
        const uint64_t w = weight44(candidate_value(s.buf[i]), c->ws);
        s.wbuf[i] = w;
        sum += w;
    }
    if (t == 0) c->n = K;
    uint64_t total;
    const uint64_t before = block_scan(sum, c->scan, total);  // (its barriers order c->n too)
    const float p = c->top_p;
    // the nucleus: the shortest prefix whose mass reaches p of the total
    if (p < 1.0f) {
        const uint64_t lo = complete ? total : c->total - c->margin, hi = complete ? total : c->total + c->margin;
        const uint64_t x_lo = scale_ceil(lo, p), x_hi = scale_ceil(hi, p);
        if (!complete && total < x_hi) {
            if (t == 0) c->n = -1;
        } else {
            uint64_t m = before;
            for (int i = i0; i < i1; ++i) {
                const uint64_t next = m + s.wbuf[i];
                // x_hi is reached first here; x_lo must be too
                if (m < x_hi && next >= x_hi) c->n = m < x_lo ? i + 1 : -1;
                m = next;
            }
        }
    } else if (!complete && t == 0) {
        c->n = -1;
    }
    __syncthreads();
    // min-p: a prefix too; the last candidate that passes ends it
    const float least = c->z_least;
    int last = -1;
    for (int i = i0; i < i1; ++i)
        if (candidate_value(s.buf[i]) >= least) last = i;
    if (last >= 0 && (last + 1 == K || candidate_value(s.buf[last + 1]) < least)) c->batch = last + 1;
    __syncthreads();
    const int n_min = c->batch;
    if (t == 0) {
        if (c->n < 0) {
            // the nucleus is not known, but min-p may cut inside the list and
            // well before the nucleus ends
            if (!complete && n_min < K) c->left = 1; else c->left = 0;
        } else if (n_min < c->n) {
            c->n = n_min;
        }
    }
    __syncthreads();
    if (c->n < 0 && c->left) {
        const uint64_t x_lo = p < 1.0f ? scale_ceil(c->total - c->margin, p) : ~0ull;
        uint64_t m = before;
        for (int i = i0; i < i1; ++i) {
            if (i == n_min - 1 && m < x_lo) c->n = n_min;  // the last kept token belongs to the nucleus
            m += s.wbuf[i];
        }
    }
    __syncthreads();
    const int n = c->n;
    if (n > 0) {
        uint64_t m = before;
        for (int i = i0; i < i1; ++i) {
            m += s.wbuf[i];
            if (i == n - 1) c->mass = m;
        }
    }
    __syncthreads();
}

// The token among the first n candidates, in vocabulary order.
template <int DT>
__device__ void pick_candidate(const RowSearchArgs& a, const Smem& s, int n, const char* row, int64_t o) {
    Ctrl* c = s.c;
    const int t = threadIdx.x;
    const uint64_t mass = c->mass;
    bool cut;
    const uint64_t target = scale_floor(mass, c->u, cut);
    if (n == 1) {
        if (t == 0) write_token<DT>(a, c, row, o, (int)(uint32_t)s.buf[0], mass);
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
                write_token<DT>(a, c, row, o, (int)i, mass);
        }
        return;
    }
    for (int i = t; i < n; i += kThreads) s.buf[i] = (s.buf[i] << 32) | (uint32_t)i;
    __syncthreads();
    sort_u64(s.buf, n);
    const int per = (n + kThreads - 1) / kThreads, i0 = min(n, t * per), i1 = min(n, i0 + per);
    uint64_t sum = 0, total;
    for (int i = i0; i < i1; ++i) sum += s.wbuf[(uint32_t)s.buf[i]];
    uint64_t m = block_scan(sum, c->scan, total);
    for (int i = i0; i < i1; ++i) {
        const uint64_t next = m + s.wbuf[(uint32_t)s.buf[i]];
        if (first ? i == 0 : (m <= target && target < next)) write_token<DT>(a, c, row, o, (int)(s.buf[i] >> 32), mass);
        m = next;
    }
}

// ---- the search over the whole row ----------------------------------------
// Every CTA of the cluster works its batches; the first one merges.

// One radix pass over the keys of a slice: bin b of the kBins gets the count
// (MASS false) or the mass (true) of the elements whose key has the bits
// `prefix` above shift + 11 and b below.  lo / hi: the two 32-bit halves.
template <int DT, bool MASS>
__device__ void radix_pass(const char* row, int64_t V, int b0, int b1, uint32_t prefix, int shift, int bits,
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
                const uint64_t w = weight44(z[e], ws);
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
__device__ void radix_pick(const Cluster& cl, const Smem& s, uint32_t prefix, int bits, uint64_t above,
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
__device__ void count_cut(const Cluster& cl, const Smem& s, const char* row, int64_t V, int b0, int b1, int k,
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
            key = kKeyNegInf + 1;
            ties = 0xffffffffu;
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
__device__ void mass_cut(const Cluster& cl, const Smem& s, const char* row, int64_t V, int b0, int b1, float p,
                         uint32_t floor_key, uint32_t floor_ties, const WeightScale& ws, uint32_t& key,
                         uint32_t& ties) {
    uint32_t* lo = reinterpret_cast<uint32_t*>(s.buf);
    const Ctrl* c0 = cl.at(s.c, 0);
    const uint64_t w_floor = floor_key > kKeyNegInf ? weight44(key_value(floor_key), ws) : 0;
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
    const uint64_t w = weight44(key_value(key), ws);  // > 0: its bin had mass
    ties = (uint32_t)((target - above + w - 1) / w);
}

// Mass of the keys above cut_key and the number of positions at it, per batch.
template <int DT>
__device__ void batch_masses(const char* row, int64_t V, int b0, int b1, uint32_t cut_key, const WeightScale& ws,
                             uint64_t* bmass, uint32_t* bties) {
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
                if (key > cut_key) m += weight44(z[e], ws);
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
    uint64_t n = 0, total;
    for (int b = b0; b < b1; ++b) n += s.bties[b];
    const uint64_t ties0 = block_scan(n, c->scan, total);
    uint64_t ties = ties0, m = 0;
    for (int b = b0; b < b1; ++b) {
        const uint64_t room = ties < cut_ties ? cut_ties - ties : 0;
        m += s.bmass[b] + min((uint64_t)s.bties[b], room) * w_tie;
        ties += s.bties[b];
    }
    uint64_t mass;
    uint64_t before = block_scan(m, c->scan, mass);
    bool cut;
    const uint64_t target = scale_floor(mass, c->u, cut);
    ties = ties0;
    for (int b = b0; b < b1; ++b) {
        const uint64_t room = ties < cut_ties ? cut_ties - ties : 0;
        const uint64_t here = s.bmass[b] + min((uint64_t)s.bties[b], room) * w_tie;
        if (before <= target && target < before + here) {
            c->batch = b;
            c->left = target - before;
            c->ties_before = (uint32_t)ties;
        }
        before += here;
        ties += s.bties[b];
    }
    if (t == 0) c->mass = mass;
    __syncthreads();
}

// One warp walks a batch in order to the element whose running kept mass
// passes `left`; returns its position and the sums on both sides of it, or -1.
template <int DT>
__device__ int walk_batch(const char* row, int64_t V, int b, uint64_t left, uint32_t cut_key, uint32_t cut_ties,
                          uint32_t ties_before, const WeightScale& ws, uint64_t& lo_side, uint64_t& hi_side) {
    constexpr int EPV = Row<DT>::EPV;
    const int lane = threadIdx.x & 31;
    uint64_t before = 0;
    uint32_t ties = ties_before;
    for (int i = 0; i < kRuns; ++i) {
        const int v = b * kBatchVecs + i * 32 + lane;
        float z[EPV];
        Row<DT>::unpack(load_vec<DT>(row, V, v), z);
        uint32_t mine = 0;
#pragma unroll
        for (int e = 0; e < EPV; ++e) mine += key_of(z[e]) == cut_key;
        uint32_t inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(DLM_FULL_MASK, inc, o);
            if (lane >= o) inc += x;
        }
        uint32_t rank = ties + inc - mine;
        ties += __shfl_sync(DLM_FULL_MASK, inc, 31);
        uint64_t w[EPV], sum = 0;
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
            const uint32_t key = key_of(z[e]);
            const bool tie = key == cut_key;
            w[e] = key > cut_key || (tie && rank < cut_ties) ? weight44(z[e], ws) : 0ull;
            rank += tie;
            sum += w[e];
        }
        uint64_t run = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t x = __shfl_up_sync(DLM_FULL_MASK, run, o);
            if (lane >= o) run += x;
        }
        uint64_t m = before + run - sum;
        int found = -1;
        uint64_t fl = 0, fh = 0;
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
            if (m <= left && left < m + w[e]) {
                found = v * EPV + e;
                fl = m;
                fh = m + w[e];
            }
            m += w[e];
        }
        before += __shfl_sync(DLM_FULL_MASK, run, 31);
        const uint32_t who = __ballot_sync(DLM_FULL_MASK, found >= 0);
        if (who) {
            const int src = __ffs(who) - 1;
            lo_side = __shfl_sync(DLM_FULL_MASK, fl, src);
            hi_side = __shfl_sync(DLM_FULL_MASK, fh, src);
            return __shfl_sync(DLM_FULL_MASK, found, src);
        }
    }
    return -1;
}

// u = 0: the first kept position of the row, whatever its weight (one warp of
// the first CTA; reads the row until it meets one).
template <int DT>
__device__ int first_kept(const char* row, int64_t V, int nb, uint32_t cut_key, uint32_t cut_ties) {
    constexpr int EPV = Row<DT>::EPV;
    const int lane = threadIdx.x & 31;
    for (int v0 = 0; v0 < nb * kBatchVecs; v0 += 32) {
        float z[EPV];
        Row<DT>::unpack(load_vec<DT>(row, V, v0 + lane), z);
        int e0 = EPV;
#pragma unroll
        for (int e = EPV - 1; e >= 0; --e) {
            const uint32_t key = key_of(z[e]);
            if (key > cut_key || (key == cut_key && cut_ties > 0)) e0 = e;
        }
        const uint32_t who = __ballot_sync(DLM_FULL_MASK, e0 < EPV);
        if (who) {
            const int src = __ffs(who) - 1;
            return (v0 + src) * EPV + __shfl_sync(DLM_FULL_MASK, e0, src);
        }
    }
    return -1;
}

// ---- the kernels -----------------------------------------------------------

template <int DT>
__device__ void write_topk(const RowSearchArgs& a, const Smem& s, int n, int64_t o) {
    for (int i = threadIdx.x; i < a.k; i += kThreads) {
        a.values[o * a.k + i] = i < n ? candidate_value(s.buf[i]) : -INFINITY;
        a.ids[o * a.k + i] = i < n ? (int32_t)(uint32_t)s.buf[i] : -1;
    }
}

template <int DT, bool SAMPLE>
__global__ void __launch_bounds__(kThreads) row_search_kernel(const RowSearchArgs a) {
    extern __shared__ __align__(16) unsigned char s_raw[];
    const int t = threadIdx.x;
    Cluster cl;
    cl.split = a.split;
    const int64_t r = blockIdx.x / a.split;
    cl.rank = (int)(blockIdx.x - r * a.split);
    const int64_t q = a.row_index ? (int64_t)a.row_index[r] : r;
    if (q < 0 || (a.n_src > 0 && q >= a.n_src)) {  // the same for every CTA of the cluster
        if (cl.rank == 0 && t == 0) raise_status(a.dev_status, DLM_DEV_BAD_INDEX);
        return;
    }
    const int64_t o = a.gather ? r : q;
    const int64_t V = a.vocab;
    const char* row = static_cast<const char*>(a.logits) + q * a.row_stride * Row<DT>::ESZ;
    constexpr int BEL = kBatchVecs * Row<DT>::EPV;  // elements of a batch
    const int nb = (int)((V + BEL - 1) / BEL);
    const int per = (nb + a.split - 1) / a.split;
    const int b0 = min(nb, cl.rank * per), b1 = min(nb, b0 + per);
    const Smem s = carve(s_raw, nb);
    Ctrl* c = s.c;

    if (t == 0) {
        float T = a.temperature, p = a.top_p, least = a.min_p;
        int k = a.k;
        bool bad = false;
        if constexpr (SAMPLE) {
            if (a.temperature_rows) T = a.temperature_rows[o];
            if (a.top_k_rows) k = a.top_k_rows[o];
            if (a.top_p_rows) p = a.top_p_rows[o];
            if (a.min_p_rows) least = a.min_p_rows[o];
            const float u = a.uniform[o];
            bad = !(T == 0.f || (T >= DLM_MIN_TEMPERATURE && T <= FLT_MAX)) || k < 0 || !(p > 0.f && p <= 1.f) ||
                  !(least >= 0.f && least <= 1.f) || !(u >= 0.f && u < 1.f);
            c->u = u;
            if (T == 0.f) k = 1, T = 1.f, p = 1.f, least = 0.f;  // the argmax
            if (k >= V) k = 0;
        }
        c->bad = bad;
        c->temperature = T;
        c->top_k = k;
        c->top_p = p;
        c->z_least = least;  // min-p until the maximum is known
        c->ws = weight_scale(0.f, bad ? 1.f : T);
        c->done = 0;
        c->count = 0;
        c->batch = 0;
    }
    __syncthreads();
    if (SAMPLE && c->bad) {
        if (cl.rank == 0 && t == 0) {
            a.token[o] = -1;
            a.prob[o] = 0.f;
            if (a.conf) a.conf[o] = 0.f;
            raise_status(a.dev_status, DLM_DEV_BAD_PARAM);
        }
        return;
    }
    // a top-k within the candidate list needs no sums; min-p alone neither
    const bool few = SAMPLE && c->top_k > 0 && c->top_k <= DLM_MAX_TOPK;
    const bool whole = V <= kCap;  // every logit fits the list
    const bool sums = !SAMPLE || (!few && !whole && (c->top_p < 1.f || c->z_least == 0.f));
    scan_rows<DT>(row, V, b0, b1, sums, c->ws.c_hi, s.sub, s.bsum);
    cl.sync();

    if (cl.rank == 0) {
        for (int rk = 1; rk < cl.split; ++rk) {  // the other slices' maxima and sums
            const int x0 = min(nb, rk * per), x1 = min(nb, x0 + per);
            const float* rs = cl.at(s.sub, rk);
            const float* rb = cl.at(s.bsum, rk);
            for (int i = x0 * kRuns + t; i < x1 * kRuns; i += kThreads) s.sub[i] = rs[i];
            if (sums)
                for (int i = x0 + t; i < x1; i += kThreads) s.bsum[i] = rb[i];
        }
        __syncthreads();
        float m = -INFINITY;
        for (int i = t; i < nb * kRuns; i += kThreads) m = max_nan(m, s.sub[i]);
        m = block_max_nan(m, c->fscan);
        if (t == 0) {
            c->ws.m = m;
            if (SAMPLE) {
                const float mp = c->z_least;
                c->z_least = mp > 0.f ? __double2float_ru((double)m + (double)c->temperature * log((double)mp)) : -INFINITY;
            }
        }
        __syncthreads();
        const WeightScale ws = c->ws;
        if (!(m > -INFINITY && m < INFINITY)) {  // NaN, +inf, or nothing but -inf
            if constexpr (SAMPLE) {
                if (t == 0) {
                    a.token[o] = -1;
                    a.prob[o] = 0.f;
                    if (a.conf) a.conf[o] = 0.f;
                }
            } else {
                write_topk<DT>(a, s, 0, o);
                if (t == 0 && a.lse) a.lse[o] = m;  // -inf, +inf or NaN
            }
            if (t == 0) {
                raise_status(a.dev_status, DLM_DEV_NONFINITE);
                c->done = 1;
            }
        } else {
            uint64_t total = 0;
            if (sums) {
                uint64_t v = 0;
                for (int b = t; b < nb; b += kThreads) {
                    const uint64_t x = batch_mass(s.sub, s.bsum, b, ws);
                    s.bmass[b] = x;
                    v += x;
                }
                block_scan(v, c->scan, total);
            }
            if constexpr (!SAMPLE) {
                if (t == 0 && a.lse)
                    a.lse[o] = m / c->temperature + logf((float)total * 5.684341886080802e-14f);
                const float least = kth_largest(s.sub, nb * kRuns, a.k, reinterpret_cast<uint32_t*>(s.buf), c);
                if (least > -INFINITY || whole) {
                    gather<DT>(row, V, 0, nb, s.sub, least, s.buf, &c->count);
                    __syncthreads();
                    const int n = (int)min(c->count, (uint32_t)0x7fffffff);
                    if (n <= kCap) {
                        sort_u64(s.buf, n);
                        write_topk<DT>(a, s, min(n, a.k), o);
                        if (t == 0) c->done = 1;
                    }
                }
            } else {
                // the sums' error, in 2^-24: 4 for each ex2 (the weight's and
                // its batch's), 2.1 per unit of exponent (three roundings),
                // whose mean over the mass is at most log2 V <= 20, 12 for
                // ten levels of additions and the products: 2^-18 in all.
                // The target and the running sum carry it each
                if (t == 0) {
                    c->total = total;
                    c->margin = (total >> 17) + nb;
                }
                const bool p_off = c->top_p >= 1.f;
                float least = -INFINITY;
                bool list = true, complete = true;
                if (few) {
                    least = kth_largest(s.sub, nb * kRuns, c->top_k, reinterpret_cast<uint32_t*>(s.buf), c);
                    list = least > -INFINITY || whole;
                } else if (whole) {
                } else if (c->top_k > 0) {
                    list = false;
                } else if (c->z_least > -INFINITY && p_off) {
                    least = c->z_least;
                } else if (!p_off) {
                    complete = false;
                    const int k0 = max(1, min(128, nb));
                    least = kth_largest(s.sub, nb * kRuns, k0, reinterpret_cast<uint32_t*>(s.buf), c);
                } else {
                    list = false;
                }
                __syncthreads();
                if (list) {
                    gather<DT>(row, V, 0, nb, s.sub, least, s.buf, &c->count);
                    __syncthreads();
                    const int n = (int)min(c->count, (uint32_t)0x7fffffff);
                    if (n <= kCap) {
                        sort_u64(s.buf, n);
                        const int k = c->top_k;
                        keep_candidates(s, k > 0 ? min(k, n) : n, complete);
                        const int kept = c->n;
                        if (kept > 0) {
                            pick_candidate<DT>(a, s, kept, row, o);
                            if (t == 0) c->done = 1;
                        }
                    }
                } else if (c->top_k == 0) {
                    // nothing is filtered: the batch sums lead to the token,
                    // if it is further than their error from a border
                    for (int b = t; b < nb; b += kThreads) s.bties[b] = 0;
                    __syncthreads();
                    find_batch(s, nb, 0, 0);
                    if (t < 32 && c->u > 0.f) {
                        uint64_t lo, hi;
                        const int tok = walk_batch<DT>(row, V, c->batch, c->left, kKeyNegInf, 0, 0, ws, lo, hi);
                        if (tok >= 0 && lo + c->margin <= c->left && c->left + c->margin < hi && t == 0) {
                            write_token<DT>(a, c, row, o, tok, c->mass);
                            c->done = 1;
                        }
                    }
                }
            }
        }
    }
    cl.sync();
    const Ctrl* c0 = cl.at(c, 0);
    const bool done = c0->done != 0;
    const WeightScale ws = c0->ws;
    const float z_least = SAMPLE ? c0->z_least : 0.f;
    cl.sync();
    if (done) return;

    // the search over the whole row
    const int k = c->top_k;
    uint32_t cut_key = kKeyNegInf, cut_ties = 0;
    if (k > 0) {
        bool list;
        count_cut<DT>(cl, s, row, V, b0, b1, k, ws, cut_key, cut_ties, list);
        if (!SAMPLE || list) {
            // the list, once more: every key from the cut on (or, when the
            // last key's ties overflow it, the keys above and the first ties)
            if (cl.rank == 0 && t == 0) c->count = 0;
            cl.sync();
            Ctrl* lead = cl.at(c, 0);
            uint64_t* dst = cl.at(s.buf, 0);
            if (list) {
                gather<DT>(row, V, b0, b1, nullptr, key_value(cut_key), dst, &lead->count);
                cl.sync();
            } else {
                gather<DT>(row, V, b0, b1, nullptr, key_value(cut_key + 1), dst, &lead->count);
                cl.sync();
                if (cl.rank == 0 && t < 32) {  // the ties in order, by one warp
                    constexpr int EPV = Row<DT>::EPV;
                    uint32_t found = 0, base = c->count;
                    for (int v0 = 0; v0 < nb * kBatchVecs && found < cut_ties; v0 += 32) {
                        float z[EPV];
                        Row<DT>::unpack(load_vec<DT>(row, V, v0 + t), z);
                        uint32_t mine = 0;
#pragma unroll
                        for (int e = 0; e < EPV; ++e) mine += key_of(z[e]) == cut_key;
                        uint32_t inc = mine;
#pragma unroll
                        for (int of = 1; of < 32; of <<= 1) {
                            const uint32_t x = __shfl_up_sync(DLM_FULL_MASK, inc, of);
                            if (t >= of) inc += x;
                        }
                        uint32_t rank = found + inc - mine;
#pragma unroll
                        for (int e = 0; e < EPV; ++e)
                            if (key_of(z[e]) == cut_key) {
                                if (rank < cut_ties) s.buf[base + rank] = candidate(z[e], (uint32_t)((v0 + t) * EPV + e));
                                ++rank;
                            }
                        found += __shfl_sync(DLM_FULL_MASK, inc, 31);
                    }
                    if (t == 0) c->count = base + min(found, cut_ties);
                }
            }
            if (cl.rank != 0) return;
            __syncthreads();
            const int n = (int)c->count;
            sort_u64(s.buf, n);
            if constexpr (!SAMPLE) {
                write_topk<DT>(a, s, min(n, k), o);
            } else {
                keep_candidates(s, min(n, k), true);
                pick_candidate<DT>(a, s, c->n, row, o);
            }
            return;
        }
    }
    if constexpr (SAMPLE) {
        if (c->top_p < 1.f) {
            uint32_t key, ties;
            mass_cut<DT>(cl, s, row, V, b0, b1, c->top_p, cut_key, cut_ties, ws, key, ties);
            cut_key = key;
            cut_ties = ties;
        }
        if (z_least > -INFINITY) {
            const uint32_t key = key_of(z_least);
            if (key > cut_key) {
                cut_key = key;
                cut_ties = 0xffffffffu;
            }
        }
        batch_masses<DT>(row, V, b0, b1, cut_key, ws, s.bmass, s.bties);
        cl.sync();
        if (cl.rank == 0) {
            for (int rk = 1; rk < cl.split; ++rk) {
                const int x0 = min(nb, rk * per), x1 = min(nb, x0 + per);
                const uint64_t* rm = cl.at(s.bmass, rk);
                const uint32_t* rt = cl.at(s.bties, rk);
                for (int i = x0 + t; i < x1; i += kThreads) {
                    s.bmass[i] = rm[i];
                    s.bties[i] = rt[i];
                }
            }
            __syncthreads();
            const uint64_t w_tie = cut_key > kKeyNegInf ? weight44(key_value(cut_key), ws) : 0;
            find_batch(s, nb, w_tie, cut_ties);
            if (t < 32) {
                uint64_t lo, hi;
                const int tok = c->u > 0.f ? walk_batch<DT>(row, V, c->batch, c->left, cut_key, cut_ties, c->ties_before,
                                                            ws, lo, hi)
                                           : first_kept<DT>(row, V, nb, cut_key, cut_ties);
                if (t == 0) write_token<DT>(a, c, row, o, max(tok, 0), c->mass);
            }
        }
        cl.sync();
    }
}

template <int DT, bool SAMPLE>
cudaError_t launch_typed(const RowSearchArgs& a, cudaStream_t st) {
    constexpr int BEL = kBatchVecs * Row<DT>::EPV;
    const size_t smem = smem_bytes((int)((a.vocab + BEL - 1) / BEL));
    if (smem > 48 * 1024) {  // the same limit whatever the call's size: calls may run side by side
        const int most = (int)smem_bytes((DLM_MAX_SEARCH_VOCAB + BEL - 1) / BEL);
        const cudaError_t e = cudaFuncSetAttribute(row_search_kernel<DT, SAMPLE>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, most);
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
    return cudaLaunchKernelEx(&cfg, row_search_kernel<DT, SAMPLE>, a);
}

template <bool SAMPLE>
cudaError_t launch(const RowSearchArgs& a, int dtype, cudaStream_t st) {
    switch (dtype) {
    case DLM_BF16: return launch_typed<DLM_BF16, SAMPLE>(a, st);
    case DLM_F16: return launch_typed<DLM_F16, SAMPLE>(a, st);
    default: return launch_typed<DLM_F32, SAMPLE>(a, st);
    }
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

cudaError_t launch_row_topk(const RowSearchArgs& a, int dtype, cudaStream_t st) { return launch<false>(a, dtype, st); }
cudaError_t launch_row_sample(const RowSearchArgs& a, int dtype, cudaStream_t st) { return launch<true>(a, dtype, st); }

}  // namespace dlm
