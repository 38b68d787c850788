// token_loss.cu -- log-probabilities of one given token per row, the clipped policy
// loss and the preference loss, with the gradients of all three by the logits.
//
// With q = softmax(z / T) and a the row's token, every loss here is a function of the
// rows' ln q_a, so that its gradient is slope / T ([v = a] - q_v), slope the loss's
// derivative by ln q_a (token_math.cuh has both).  `state` holds what the gradient
// needs of a row: maximum, 1 / sum, 1 - q_a, slope.
//
// All of it is bound by HBM: the sums by one read of the row, the gradient by a read and
// a write.  One kernel does sums, gradient or both:
//  * A row is cut over a cluster of 1 to 8 CTAs.  Clusters stay and take the next row that
//    has not begun from the hardware (a cluster launch cancelled in their favour), so rows
//    that are not read cost nothing and no counter is needed.
//  * In each CTA one thread fetches: 16 KB at a time into a ring with asynchronous bulk
//    copies, across rows, so that HBM does not wait at a row's end.  Eight warps add up
//    what is there.  A warp of its own merges the cluster's shares (sent into shared memory,
//    counted by a barrier there) and works out the loss, while the others go on.
//  * A step reads a row once: the slice stays in the ring (up to 96 KB) from its sums to
//    its gradient.  Rows above 768 KB come twice.
// Measured (GB300, a call among others; HBM copies 6.8 TB/s):
//    2048 rows of 152064 bf16: log-probabilities 94 us (6.6 TB/s of 623 MB);
//      policy step, a quarter of the rows without a loss, 184 us (5.9 TB/s of 1.09 GB);
//      gradient alone 187 us (6.7 TB/s of 1.25 GB)
//    512 rows of 126464 bf16: policy loss 30 us, step with a quarter unread 48 us: of
//      either about 9 us are there whatever the size (the launch, the first copies, the
//      last row's exchange; 32 rows of 1024 take 6 us)
//    A step's row in the cluster, slices of 76 KB, in cycles: sums 5500 (the copies), shares
//      1100, merge and loss 1800, gradient 4400.  With the loss in 64-bit arithmetic 2300, with
//      one of the eight warps doing it too every row took 2 us more.
// Without these: a CTA per row, loads to registers, step 837 us; chunks of 8 KB 109 us for
// the log-probabilities, two CTAs per SM 101, four of half the threads 102; the next row's
// sums taken before a row's gradient where the row then comes twice, 197 us for the step; a
// maximum saved per vector (a reference kept until a weight passes 2^90) 103 us for the
// log-probabilities.
// The preference step is two launches, since a gradient needs its whole pair: sums, and
// gradients, whose launch adds up the pairs.  1024 rows of 126464 bf16 in 8 pairs: 128 us, 50
// and 76 alone; floor 76 us with one read of the rows, 114 with two.  One launch, rows
// handed out by a counter, each pair's gradients as soon as its sums were there: 140 us;
// the second read came from HBM there too.
#include "common.cuh"
#include "launch.h"
#include "row_vec.cuh"
#include "token_math.cuh"

namespace dlm {

namespace {

constexpr int kThreads = kRowThreads;   // consumers: threads that do the arithmetic
constexpr int kWarps = kRowWarps;
constexpr int kBlock = kThreads + 64;   // and the warps that finish rows and that fetch them
constexpr int kPerThread = 4;           // vectors of a chunk per thread
constexpr int kChunkVecs = kPerThread * kThreads, kChunkBytes = kChunkVecs * 16;
constexpr int kItems = 4;               // rows that the fetching warp may be ahead
constexpr int kSlots = 8;               // rows whose shares may be on their way (more than kItems + 2)
// CTAs per SM, and the chunks that each has room for: a step's slices want room, sums or a
// gradient alone more warps (2048 x 152064 bf16: log-probabilities 97 us with three, 101 with
// two; policy step 191 with three, 184 with two).
template <bool SUMS, bool GRAD>
struct Shape {
    static constexpr int ctas = SUMS && GRAD ? 2 : 3, ring = SUMS && GRAD ? 6 : 4;
};
constexpr int kMaxRing = 6;
constexpr float kRebase = 12.0f;        // powers of 2 of headroom before a thread's reference moves
// Rows' bytes that a preference step leaves in L2 for its gradient (1024 rows of 126464
// bf16: 132 us with 60 to 80 MB, 134 with 40, 139 without, 143 with the first rows first).
constexpr int64_t kStays = 70 << 20;
constexpr int kLeast = 8 * 1024;        // a slice is not cut below this to fill the GPU
constexpr long long kWaitLimit = 4000000000LL;  // ~2 s

// What a thread, a warp or a CTA knows of a row: the sum of its slice's weights
// 2^((z - ref) c), without the token's, relative to the largest logit of them; and the
// token's logit (-inf: it lies in another slice).
struct __align__(16) Part {
    float ref, sum, z, pad;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(DLM_FULL_MASK, v, o);
    return v;
}
// The sum over the lanes in a fixed order, in all lanes.
__device__ __forceinline__ Part warp_part(Part a, float c) {
    Part b;
    b.ref = warp_max_nan(a.ref);
    b.z = warp_max_nan(a.z);
    b.sum = warp_sum(a.sum * ex2((a.ref - or_zero(b.ref)) * c));
    b.pad = 0.f;
    return b;
}

// ---- barriers and copies ------------------------------------------------------

__device__ __forceinline__ void arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ uint32_t remote(const void* p, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void arrive_at(uint64_t* bar, int rank) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote(bar, rank)) : "memory");
}
// Waits for a phase; false if that takes too long.  CLUSTER: other CTAs write what it
// stands for.
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity) {
    long long t0 = 0;
    for (int n = 0;; ++n) {
        uint32_t ok;
        if (CLUSTER)
            asm volatile(
                "{\n\t.reg .pred p;\n\t"
                "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(ok)
                : "r"(smem_u32(bar)), "r"(parity)
                : "memory");
        else
            ok = mbar_try_wait(bar, parity);
        if (ok) return true;
        if (n == 0)
            t0 = clock64();
        else if (clock64() - t0 > kWaitLimit)
            return false;
    }
}
// The same for a whole warp, whose lanes go on together or give up together.
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) {
    return __all_sync(DLM_FULL_MASK, wait_for<CLUSTER>(bar, parity));
}
// A share into CTA `rank`'s slot, counted there by its barrier.
__device__ __forceinline__ void send(Part* slot, uint64_t* bar, int rank, Part p) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                     remote(slot, rank)),
                 "r"(__float_as_uint(p.ref)), "r"(__float_as_uint(p.sum)), "r"(__float_as_uint(p.z)), "r"(0u),
                 "r"(remote(bar, rank))
                 : "memory");
}
// How long L2 keeps what a copy reads.
__device__ __forceinline__ uint64_t l2_normal() {
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ uint64_t l2_stays() {
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ uint64_t l2_goes() {
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
// Untiled copy into this CTA's shared memory: both addresses and the size in whole 16 bytes.
__device__ __forceinline__ void fetch(void* dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t policy) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
                 : "memory");
}
// Every launch here may begin while the one before it on the stream ends, and nothing of
// it touches memory before that has ended.
__device__ __forceinline__ void wait_prior() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Asks for a cluster of the grid that has not started: its first CTA's index arrives
// in all CTAs of this one, or that there is none.
__device__ __forceinline__ void ask_next(void* answer, uint64_t* bar, bool cluster) {
    if (cluster)
        asm volatile(
            "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.multicast::cluster::all.b128 [%0], "
            "[%1];" ::"r"(smem_u32(answer)),
            "r"(smem_u32(bar))
            : "memory");
    else
        asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                         smem_u32(answer)),
                     "r"(smem_u32(bar))
                     : "memory");
}
__device__ __forceinline__ bool next_cta(const void* answer, uint32_t& cta) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 a;\n\t"
        "ld.shared.b128 a, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n\t}"
        : "=r"(ok), "=r"(cta)
        : "r"(smem_u32(answer))
        : "memory");
    return ok != 0;
}

// Element e of a vector replaced by the bits x.
template <int DT>
__device__ __forceinline__ uint4 with_elem(uint4 w, int e, uint32_t x) {
    uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == DLM_F32) {
            if (i == e) r[i] = x;
        } else {
            if (i == e >> 1) r[i] = e & 1 ? (r[i] & 0xffffu) | x << 16 : (r[i] & 0xffff0000u) | x;
        }
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}
template <int DT>
__device__ constexpr uint32_t neg_inf_bits() {
    if constexpr (DT == DLM_F32)
        return 0xff800000u;
    else
        return Row<DT>::kNegInf;
}
// ---- rows -----------------------------------------------------------------------

// A row as the fetching warp hands it over.
enum : int { kEnd, kSkip, kNone, kRow };  // no more rows; not touched; without a loss or gradient; read
struct Item {
    int64_t q, o;     // its place in the logits, and in the per-row arrays
    int kind, token;
    float weight;
    float m, inv, away, k;  // gradient from the state
};

struct Shared {
    Part part[kSlots][8 * kWarps];  // every warp's of every CTA of the cluster
    Item item[kItems];
    float4 row[kItems];             // maximum, 1 / sum, 1 - q of the token, slope
    uint64_t item_full[kItems], item_empty[kItems];
    uint64_t full[kMaxRing], empty[kMaxRing];
    uint64_t shares[kSlots], row_ready[kItems];
    uint64_t next, next_free;       // the answer to ask_next is there; every CTA has read it (in the first CTA)
    __align__(16) unsigned char answer[16];
};
__host__ __device__ inline size_t ring_offset() { return (sizeof(Shared) + 127) & ~(size_t)127; }

// Position in the ring of chunks, and the parity of its full barrier.
struct Cursor {
    int at = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void step(int n) {
        if (++at == n) {
            at = 0;
            parity ^= 1u;
        }
    }
};

template <int DT>
struct TokenSlice {
    int v0, n;        // vectors of this CTA
    int whole;        // those that V does not cut
    int chunks, most_chunks;  // its chunks; the most that a CTA of the cluster has
    __device__ TokenSlice(int64_t V, int split, int rank) {
        constexpr int EPV = Row<DT>::EPV;
        const int nv = (int)((V + EPV - 1) / EPV);
        const int per = ((nv + split - 1) / split + 7) & ~7;
        v0 = min(nv, rank * per);
        n = min(nv, v0 + per) - v0;
        whole = max(0, min((int)(V / EPV), v0 + n) - v0);
        chunks = (whole + kChunkVecs - 1) / kChunkVecs;
        most_chunks = (per + kChunkVecs - 1) / kChunkVecs;
    }
};

// Running sum of a thread.
struct Running {
    float ref = -FLT_MAX;  // of the weights
    float top = -INFINITY; // the largest logit so far
    f2 sum = pack2(0.f, 0.f);
};
template <int DT, int N>
__device__ __forceinline__ void add_vectors(Running& a, const uint4 (&w)[N], f2 c2, f2 lo2, float c) {
    constexpr int EPV = Row<DT>::EPV;
    float m = Row<DT>::vmax(w[0]);
#pragma unroll
    for (int u = 1; u < N; ++u) m = max_nan(m, Row<DT>::vmax(w[u]));
    a.top = max_nan(a.top, m);
    if ((m - a.ref) * c > kRebase) {
        const float e = ex2((a.ref - m) * c);
        a.sum = mul2(a.sum, pack2(e, e));
        a.ref = m;
    }
    const f2 r2 = pack2(a.ref, a.ref);
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
    a.sum = add2(a.sum, sum[0]);
}

__device__ __forceinline__ Temper temper(const TokenArgs& a) { return Temper{a.scale, a.scale_lo, Two{a.inv_t, a.inv_t_lo}}; }

// What a row's loss needs beside its sums.
struct RowInputs {
    float weight, advantage, old_logp, ref_logp;
};
__device__ __forceinline__ RowInputs row_inputs(const TokenArgs& a, int64_t o, float weight) {
    return RowInputs{weight, a.op == kTokenPolicy ? a.advantages[o] : 0.f, a.old_logp ? a.old_logp[o] : 0.f,
                     a.ref_logp ? a.ref_logp[o] : 0.f};
}
// What a row's loss is.
__device__ __forceinline__ LossSlope row_loss(const TokenArgs& a, const TokenRow& t, const RowInputs& in) {
    if (a.op == kTokenPolicy)
        return policy_row(a.policy, t.logp, in.weight, in.advantage, a.old_logp != nullptr, in.old_logp, in.ref_logp);
    return LossSlope{0.f, in.weight};
}
// Its outputs, by one thread.
__device__ __forceinline__ void write_row(const TokenArgs& a, int64_t o, const TokenRow& t, const RowInputs& in, LossSlope x) {
    if (!t.ok || x.slope != x.slope) raise_status(a.dev_status, DLM_DEV_NONFINITE);
    if (a.op == kTokenPolicy) a.loss[o] = x.loss;
    if (a.logp) a.logp[o] = rounded(t.logp);
    if (a.lse) a.lse[o] = token_lse(t, temper(a));
    if (a.state) {
        const double term = a.op == kTokenPreference ? (double)in.weight * (((double)t.logp.hi - (double)in.ref_logp) + (double)t.logp.lo) : 0.0;
        float4* s = reinterpret_cast<float4*>(a.state + o * DLM_TOKEN_STATE);
        // (preference: the pair's slope is still to come; 0 stands for a row in no pair)
        s[0] = make_float4(t.m, t.inv, t.away, a.op == kTokenPreference && !a.paired ? 0.f : x.slope);
        s[1] = make_float4(__int_as_float(__double2loint(term)), __int_as_float(__double2hiint(term)), __int_as_float(-1), 0.f);
    }
}
// A row without a loss.
__device__ void finish_none(const TokenArgs& a, int64_t o) {
    if (a.op == kTokenPolicy) a.loss[o] = 0.f;
    if (a.logp) a.logp[o] = 0.f;
    if (a.lse) a.lse[o] = 0.f;
    if (a.state) {
        float4* s = reinterpret_cast<float4*>(a.state + o * DLM_TOKEN_STATE);
        s[0] = make_float4(0.f, 0.f, 0.f, 0.f);
        s[1] = make_float4(0.f, 0.f, __int_as_float(-1), 0.f);
    }
}

// A row's shares of all CTAs of the cluster, in slot s, and what follows from them.
__device__ __forceinline__ TokenRow merge_row(const TokenArgs& a, const Shared& sh, int s, int n) {
    const int lane = threadIdx.x & 31;
    const float c = a.scale;
    Part p = lane < n ? sh.part[s][lane] : Part{-INFINITY, 0.f, -INFINITY, 0.f};
    if (lane + 32 < n) {
        const Part b = sh.part[s][lane + 32];
        const float ref = max_nan(p.ref, b.ref), to = or_zero(ref);
        p.sum = p.sum * ex2((p.ref - to) * c) + b.sum * ex2((b.ref - to) * c);
        p.ref = ref;
        p.z = max_nan(p.z, b.z);
    }
    p = warp_part(p, c);
    return token_row(p.ref, p.sum, p.z, temper(a));
}

// The fetching warp's thread: rows in the order in which the hardware gives them, their
// settings, and their slices chunk by chunk into the ring.  What the next row needs is
// asked for while this row's chunks are on their way: the row itself (about 1 us), then
// its token and weight (another), which are not looked at before the row's turn.
template <int DT, bool SUMS, bool GRAD>
struct Fetcher {
    const TokenArgs& a;
    Shared& sh;
    unsigned char* ring;
    const int rank;
    const TokenSlice<DT> sl;
    Cursor cur;
    uint32_t issued = 0;
    Item next_item{};
    uint32_t asked = 0, answers = 0;     // (asked: the first CTA's)
    bool have_next = false;                      // next_item is being read

    __device__ Fetcher(const TokenArgs& args, Shared& s, unsigned char* r, int k)
        : a(args), sh(s), ring(r), rank(k), sl(args.vocab, args.split, k) {}

    // (a preference step's gradient: the last rows first, which L2 still has)
    __device__ __forceinline__ int64_t row_of(uint32_t cta) const {
        const int64_t r = cta / a.split;
        return !SUMS && a.paired ? a.n_rows - 1 - r : r;
    }
    // Starts to read what belongs to row r.
    __device__ __forceinline__ void read_row(int64_t r) {
        Item& it = next_item;
        it.kind = kRow;
        it.q = r;
        if (SUMS && a.row_index) {
            it.q = a.row_index[r];
            if (it.q < 0 || (a.n_src > 0 && it.q >= a.n_src)) {
                it.kind = kSkip;
                if (rank == 0) raise_status(a.dev_status, DLM_DEV_BAD_INDEX);
            }
        }
        it.o = a.gather ? r : it.q;
        if (it.kind == kSkip) return;
        it.token = a.tokens[it.o];
        if (SUMS) {
            it.weight = a.weights ? a.weights[it.o] : 1.f;
        } else {
            const float4 s = *reinterpret_cast<const float4*>(a.state + r * DLM_TOKEN_STATE);
            it.m = s.x;
            it.inv = s.y;
            it.away = s.z;
            it.k = s.w;
            it.weight = 1.f;
            if (a.grad_loss) {
                const int64_t at = a.op == kTokenPreference ? (int64_t)__float_as_int(a.state[r * DLM_TOKEN_STATE + 6]) : r;
                it.weight = at >= 0 && at < a.n_up ? a.grad_loss[at] : 0.f;
            }
        }
    }
    // The item that read_row() began.
    __device__ __forceinline__ Item row_read() {
        Item it = next_item;
        if (it.kind == kRow) {
            bool none = it.token < 0 || it.token >= a.vocab;
            if (SUMS) {
                none = none || it.weight == 0.f;
                if (it.token >= a.vocab && rank == 0) raise_status(a.dev_status, DLM_DEV_BAD_INDEX);
            } else {
                it.k *= a.inv_t * it.weight;
                none = none || it.k == 0.f || it.inv == 0.f;
            }
            if (none) it.kind = kNone;
        }
        return it;
    }
    // The first CTA asks for a row once every CTA has read the last answer.
    __device__ __forceinline__ bool ask(bool block) {
        if (rank != 0 || asked > answers) return true;
        if (asked > 0) {
            const uint32_t parity = (asked - 1) & 1u;
            if (block ? !wait_for<true>(&sh.next_free, parity) : !mbar_test_wait(&sh.next_free, parity)) return !block;
        }
        ask_next(sh.answer, &sh.next, a.split > 1);
        ++asked;
        return true;
    }
    // Takes the answer if it is there (block: waits for it).
    __device__ __forceinline__ bool look_ahead(bool block) {
        if (have_next) return ask(false);
        if (!ask(block)) return false;
        if (block ? !wait_for<true>(&sh.next, answers & 1u) : !mbar_test_wait(&sh.next, answers & 1u)) return !block;
        uint32_t cta;
        const bool more = next_cta(sh.answer, cta);
        ++answers;
        have_next = true;
        if (!more) {
            next_item.kind = kEnd;
            asked = answers + 1;  // and nothing is asked for any more
            return true;
        }
        mbar_expect_tx(&sh.next, 16);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the answer has been read before the next one is written
        arrive_at(&sh.next_free, 0);
        read_row(row_of(cta));
        return ask(false);
    }
    __device__ bool run() {
        const int passes = SUMS && GRAD && !a.resident ? 2 : 1;
        read_row(row_of(blockIdx.x));
        for (uint32_t i = 0;; ++i) {
            const Item it = row_read();
            have_next = false;
            const int slot = i % kItems;
            if (!wait_for(&sh.item_empty[slot], ((i / kItems) & 1u) ^ 1u)) return false;
            sh.item[slot] = it;
            arrive(&sh.item_full[slot]);
            if (it.kind == kEnd) return true;
            if (it.kind == kRow) {
                // a preference step's gradient begins with the rows whose sums came last
                const uint64_t policy = !a.paired ? l2_normal() : SUMS && it.q >= a.stay_from ? l2_stays() : l2_goes();
                const char* src = static_cast<const char*>(a.logits) + it.q * a.row_stride * Row<DT>::ESZ + (int64_t)sl.v0 * 16;
                for (int pass = 0; pass < passes; ++pass)
                    for (int c = 0; c < sl.chunks; ++c) {
                        if (!wait_for(&sh.empty[cur.at], cur.parity ^ 1u)) return false;
                        const uint32_t bytes = (uint32_t)min(kChunkVecs, sl.whole - c * kChunkVecs) * 16;
                        mbar_expect_tx(&sh.full[cur.at], bytes);
                        fetch(ring + cur.at * kChunkBytes, src + (int64_t)c * kChunkBytes, bytes, &sh.full[cur.at], policy);
                        cur.step(a.ring);
                        ++issued;
                        look_ahead(false);
                    }
            }
            if (!have_next && !look_ahead(true)) return false;
        }
    }
    // Copies still in flight land before the CTA ends.
    __device__ void drain() {
        Cursor c;
        for (uint32_t i = 0; i < issued; ++i) {
            if (i + a.ring >= issued) wait_for(&sh.full[c.at], c.parity);
            c.step(a.ring);
        }
        wait_for<true>(&sh.next, answers & 1u);
    }
};

// Zeros where a row has no gradient.
template <int DT>
__device__ void write_zeros(char* out, int64_t V, const TokenSlice<DT>& sl) {
    const int t = threadIdx.x;
    uint4* dst = reinterpret_cast<uint4*>(out) + sl.v0;
    for (int v = t; v < sl.whole; v += kThreads) st_row(dst + v, make_uint4(0, 0, 0, 0));
    if (sl.whole < sl.n)
        for (int64_t e = (int64_t)(sl.v0 + sl.whole) * Row<DT>::EPV + t; e < V; e += kThreads) store_elem<DT>(out, e, 0.f);
}

// ---- pairs --------------------------------------------------------------------------

// The loss of pair i from its scores.
__device__ __forceinline__ LossSlope pair_loss(const TokenArgs& a, int64_t i, double chosen, double rejected) {
    return preference_pair(a.preference, chosen, rejected, a.margins ? a.margins[i] : 0.f,
                           a.pair_weights ? a.pair_weights[i] : 1.f);
}
// Its outputs, by one thread: its slope.
__device__ float finish_pair(const TokenArgs& a, int64_t i, double chosen, double rejected) {
    const LossSlope x = pair_loss(a, i, chosen, rejected);
    a.loss[i] = x.loss;
    if (a.score) {
        a.score[2 * i] = (float)chosen;
        a.score[2 * i + 1] = (float)rejected;
    }
    if (x.slope != x.slope) raise_status(a.dev_status, DLM_DEV_NONFINITE);
    return x.slope;
}

// The offsets put right (within the rows and in order) for a preference step's second
// launch, by one warp of the first.
__device__ void clean_offsets(const TokenArgs& a) {
    const int lane = threadIdx.x & 31;
    const int64_t n = 2 * a.n_pairs + 1;
    int32_t top = 0;
    for (int64_t base = 0; base < n; base += 32) {
        const int64_t i = base + lane;
        const int32_t given = i < n ? a.offsets[i] : 0;
        int32_t x = (int32_t)min((int64_t)max(given, 0), a.n_rows);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t y = __shfl_up_sync(DLM_FULL_MASK, x, o);
            if (lane >= o) x = max(x, y);
        }
        x = max(x, top);
        top = __shfl_sync(DLM_FULL_MASK, x, 31);
        if (i < n) {
            a.at[i] = x;
            if (x != given) raise_status(a.dev_status, DLM_DEV_BAD_INDEX);
        }
    }
}

// The pair of a row, by a warp: its rows [from, to), those of the sequence that is not
// preferred from `mid` on, and its slope.  Rows in no pair: pair -1, slope 0.
struct PairOf {
    int64_t pair = -1, from = 0, mid = 0, to = 0;
    double score[2] = {0.0, 0.0};
    float slope = 0.f;
};
__device__ __noinline__ PairOf pair_of(const TokenArgs& a, int64_t r) {
    const int lane = threadIdx.x & 31;
    const int64_t n = 2 * a.n_pairs;
    PairOf p;
    p.to = a.n_rows;
    if (n == 0) return p;
    const int64_t first = a.at[0], last = a.at[n];
    if (r < first || r >= last) {
        p.from = r < first ? 0 : last;
        p.to = r < first ? first : a.n_rows;
        return p;
    }
    int64_t lo = 0, hi = n;  // the last sequence that begins at or before r, 32 places at a time
    while (hi - lo > 1) {
        const int64_t step = (hi - lo + 31) / 32, i = lo + lane * step;
        const uint32_t at_or_before = __ballot_sync(DLM_FULL_MASK, i < hi && a.at[i] <= r);
        lo += (__popc(at_or_before) - 1) * step;
        hi = min(hi, lo + step);
    }
    p.pair = lo >> 1;
    p.from = a.at[2 * p.pair];
    p.mid = a.at[2 * p.pair + 1];
    p.to = a.at[2 * p.pair + 2];
#pragma unroll 8
    for (int64_t k = p.from + lane; k < p.to; k += 32) {
        const double term = *reinterpret_cast<const double*>(a.state + k * DLM_TOKEN_STATE + 4);
        p.score[0] += k < p.mid ? term : 0.0;
        p.score[1] += k < p.mid ? 0.0 : term;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        p.score[0] += __shfl_xor_sync(DLM_FULL_MASK, p.score[0], o);
        p.score[1] += __shfl_xor_sync(DLM_FULL_MASK, p.score[1], o);
    }
    p.slope = pair_loss(a, p.pair, p.score[0], p.score[1]).slope;
    return p;
}

// A preference step's second launch: the warp that finishes sums in the first finds the
// slope of each row's pair, ahead of the warps that write the gradient.  (A pair is added
// up once by every CTA that has rows of it, in one order; the first row's cluster writes
// its loss.)
__device__ bool find_slopes(const TokenArgs& a, Shared& sh, int rank) {
    const int lane = threadIdx.x & 31;
    PairOf p;
    uint32_t rows = 0;
    for (uint32_t i = 0;; ++i) {
        const int slot = i % kItems;
        if (!wait_warp(&sh.item_full[slot], (i / kItems) & 1u)) return false;
        const int kind = sh.item[slot].kind;
        const int64_t r = sh.item[slot].o;
        if (kind == kEnd) return true;
        if (r < p.from || r >= p.to) p = pair_of(a, r);
        if (kind == kRow) {
            if (lane == 0) {
                sh.row[rows % kItems].w = r >= p.mid ? -p.slope : p.slope;
                arrive(&sh.row_ready[rows % kItems]);
            }
            ++rows;
        }
        if (rank == 0 && lane == 0) {
            if (p.pair >= 0 && r == p.from) finish_pair(a, p.pair, p.score[0], p.score[1]);
            for (int64_t k = r; k < a.n_pairs; k += a.n_rows)  // pairs without rows
                if (a.at[2 * k] == a.at[2 * k + 2]) finish_pair(a, k, 0.0, 0.0);
        }
        __syncwarp();
        if (lane == 0) arrive(&sh.item_empty[slot]);
    }
}

// A warp of its own finishes the rows: it waits for all CTAs' shares, merges them and
// works the loss out, while the others go on.  With a gradient every CTA's does, to go on
// with the slope; the first CTA's writes.
template <bool GRAD>
__device__ bool finish_rows(const TokenArgs& a, Shared& sh, int rank) {
    const int lane = threadIdx.x & 31, n_parts = a.split * kWarps;
    uint32_t rows = 0;
    for (uint32_t i = 0;; ++i) {
        const int slot = i % kItems;
        if (!wait_warp(&sh.item_full[slot], (i / kItems) & 1u)) return false;
        const int kind = sh.item[slot].kind;
        const int64_t o = sh.item[slot].o;
        if (kind == kEnd) return true;
        if (kind == kNone && rank == 0 && lane == 0) finish_none(a, o);
        if (kind == kRow) {
            if (GRAD || rank == 0) {
                const RowInputs in = row_inputs(a, o, sh.item[slot].weight);
                const int ps = rows % kSlots;
                if (lane == 0) mbar_expect_tx(&sh.shares[ps], n_parts * (uint32_t)sizeof(Part));
                if (!wait_warp<true>(&sh.shares[ps], (rows / kSlots) & 1u)) return false;
                const TokenRow x = merge_row(a, sh, ps, n_parts);
                const LossSlope y = row_loss(a, x, in);
                if (GRAD && lane == 0) {  // first of all: the gradient waits for it
                    sh.row[rows % kItems] = make_float4(x.m, x.inv, x.away, y.slope);
                    arrive(&sh.row_ready[rows % kItems]);
                }
                if (rank == 0 && lane == 0) write_row(a, o, x, in, y);
            }
            ++rows;
        }
        if (!GRAD && a.paired && a.n_pairs > 0 && rank == 0 && o == 0) clean_offsets(a);
        __syncwarp();
        if (lane == 0) arrive(&sh.item_empty[slot]);
    }
}

// The sums of this CTA's slice of row q, the chunks freed as they are done with where they
// are not used again; false if they do not come.
template <int DT>
__device__ __forceinline__ bool take_sums(const TokenArgs& a, Shared& sh, unsigned char* ring, const TokenSlice<DT>& sl,
                                          int64_t q, int token, bool keep, Cursor& cur, Part& part) {
    constexpr int EPV = Row<DT>::EPV;
    const int t = threadIdx.x, lane = t & 31;
    const float c = a.scale;
    const f2 c2 = pack2(c, c), lo2 = pack2(a.scale_lo, a.scale_lo);
    const int tv = token / EPV - sl.v0;  // the token's vector in the slice
    const bool mine = tv >= 0 && tv < sl.n && (tv & (kThreads - 1)) == t;
    Running s;
    float z_token = -INFINITY;
    for (int ch = 0; ch < sl.chunks; ++ch) {
        if (!wait_warp(&sh.full[cur.at], cur.parity)) return false;
        uint4* data = reinterpret_cast<uint4*>(ring + cur.at * kChunkBytes);
        const int base = ch * kChunkVecs, n = min(kChunkVecs, sl.whole - base);
        if (mine && tv >= base && tv < base + n) {  // the token leaves the slice (its vector is this thread's)
            z_token = Row<DT>::scalar(data + (tv - base), token % EPV);
            data[tv - base] = with_elem<DT>(data[tv - base], token % EPV, neg_inf_bits<DT>());
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before a copy writes here again
        }
        if (n == kChunkVecs) {
            uint4 w[kPerThread];
#pragma unroll
            for (int u = 0; u < kPerThread; ++u) w[u] = data[t + u * kThreads];
            add_vectors<DT>(s, w, c2, lo2, c);
        } else {
            for (int v = t; v < n; v += kThreads) {
                const uint4 w[1] = {data[v]};
                add_vectors<DT>(s, w, c2, lo2, c);
            }
        }
        if (!keep) {
            __syncwarp();
            if (lane == 0) arrive(&sh.empty[cur.at]);
        }
        cur.step(a.ring);
    }
    if (sl.whole < sl.n && (sl.whole & (kThreads - 1)) == t) {  // the row's last, cut vector
        const char* row = static_cast<const char*>(a.logits) + q * a.row_stride * Row<DT>::ESZ;
        uint4 w[1] = {load_vec<DT>(row, a.vocab, sl.v0 + sl.whole)};
        if (mine && tv == sl.whole) {
            z_token = Row<DT>::scalar(row, token);
            w[0] = with_elem<DT>(w[0], token % EPV, neg_inf_bits<DT>());
        }
        add_vectors<DT>(s, w, c2, lo2, c);
    }
    part = warp_part(Part{s.top, hsum2(s.sum) * ex2((s.ref - or_zero(s.top)) * c), z_token, 0.f}, c);
    return true;
}

// k ([v = token] - q_v) over this CTA's slice of row q.
struct RowSlope {
    float m, inv, away, k;
};
template <int DT>
__device__ __forceinline__ bool put_gradient(const TokenArgs& a, Shared& sh, unsigned char* ring, const TokenSlice<DT>& sl,
                                             int64_t q, int token, RowSlope x, bool there, Cursor& from) {
    constexpr int EPV = Row<DT>::EPV;
    const int t = threadIdx.x, lane = t & 31;
    const float c = a.scale;
    char* out = static_cast<char*>(a.grad) + q * a.grad_stride * Row<DT>::ESZ;
    if (x.k == 0.f) {  // a clipped row, or one of no pair: zeros, whatever the row holds
        for (int ch = 0; ch < sl.chunks; ++ch) {
            if (!there && !wait_warp(&sh.full[from.at], from.parity)) return false;
            if (lane == 0) arrive(&sh.empty[from.at]);
            from.step(a.ring);
        }
        write_zeros<DT>(out, a.vocab, sl);
        return true;
    }
    const Slope slope(x.m, c, -x.k * x.inv);
    uint4* dst = reinterpret_cast<uint4*>(out) + sl.v0;
    for (int ch = 0; ch < sl.chunks; ++ch) {
        if (!there && !wait_warp(&sh.full[from.at], from.parity)) return false;
        const uint4* data = reinterpret_cast<const uint4*>(ring + from.at * kChunkBytes);
        const int base = ch * kChunkVecs, n = min(kChunkVecs, sl.whole - base);
        if (n == kChunkVecs) {
#pragma unroll
            for (int u = 0; u < kPerThread; ++u)
                st_row(dst + base + t + u * kThreads, slope_of<DT>(data[t + u * kThreads], slope));
        } else {
            for (int v = t; v < n; v += kThreads) st_row(dst + base + v, slope_of<DT>(data[v], slope));
        }
        __syncwarp();
        if (lane == 0) arrive(&sh.empty[from.at]);
        from.step(a.ring);
    }
    if (sl.whole < sl.n && (sl.whole & (kThreads - 1)) == t) {
        const char* row = static_cast<const char*>(a.logits) + q * a.row_stride * Row<DT>::ESZ;
        for (int64_t e = (int64_t)(sl.v0 + sl.whole) * EPV; e < a.vocab; ++e)
            store_elem<DT>(out, e, -x.k * x.inv * ex2((Row<DT>::scalar(row, e) - x.m) * c));
    }
    const int tv = token / EPV - sl.v0;
    if (tv >= 0 && tv < sl.n && (tv & (kThreads - 1)) == t) store_elem<DT>(out, token, x.k * x.away);  // (after this thread's own vector)
    return true;
}

// The arithmetic's warps.  A row's slope is known about 2 us after its sums (to all CTAs and
// back): where the ring holds two slices a step takes the next row's sums before a row's
// gradient (2048 rows of 16000 bf16: 33 us without).
template <int DT, bool SUMS, bool GRAD>
__device__ bool work_rows(const TokenArgs& a, Shared& sh, unsigned char* ring, int rank) {
    constexpr bool BOTH = SUMS && GRAD;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const TokenSlice<DT> sl(a.vocab, a.split, rank);
    const bool there = BOTH && a.resident;
    const bool ahead = there && 2 * sl.most_chunks <= a.ring;
    Cursor cur;
    uint32_t rows = 0;      // rows whose sums were taken
    int64_t open_q = -1;    // a row before whose gradient is still to come, its token, its place in the ring
    int open_token = 0;
    Cursor open_from;
    // the gradient of a row (its number) from the slope that the finishing warp leaves
    auto gradient = [&](uint32_t row, int64_t q, int token, Cursor& from) -> bool {
        const int rs = row % kItems;
        if (!wait_warp(&sh.row_ready[rs], (row / kItems) & 1u)) return false;
        const float4 y = sh.row[rs];
        return put_gradient<DT>(a, sh, ring, sl, q, token, RowSlope{y.x, y.y, y.z, y.w * a.inv_t}, there, from);
    };
    for (uint32_t i = 0;; ++i) {
        const int slot = i % kItems;
        if (!wait_warp(&sh.item_full[slot], (i / kItems) & 1u)) return false;
        const Item& it = sh.item[slot];
        const int kind = it.kind, token = it.token;
        const int64_t q = it.q;
        if (GRAD && kind == kNone)
            write_zeros<DT>(static_cast<char*>(a.grad) + q * a.grad_stride * Row<DT>::ESZ, a.vocab, sl);
        Cursor from = cur;
        if (SUMS && kind == kRow) {
            Part part;
            if (!take_sums<DT>(a, sh, ring, sl, q, token, there, cur, part)) return false;
            const int ps = rows % kSlots, to = GRAD ? a.split : 1;  // every CTA, or the first
            if (lane < to) send(&sh.part[ps][rank * kWarps + warp], &sh.shares[ps], lane, part);
        }
        if (BOTH) {
            if (open_q >= 0 && (kind == kRow || kind == kEnd)) {
                if (!gradient(rows - 1, open_q, open_token, open_from)) return false;
                open_q = -1;
            }
            if (kind == kRow) {
                if (ahead) {
                    open_q = q;
                    open_token = token;
                    open_from = from;
                } else if (!gradient(rows, q, token, there ? from : cur)) {
                    return false;
                }
            }
        } else if (GRAD && kind == kRow) {
            RowSlope x{it.m, it.inv, it.away, it.k};
            if (a.paired) {
                const int rs = rows % kItems;
                if (!wait_warp(&sh.row_ready[rs], (rows / kItems) & 1u)) return false;
                x.k *= sh.row[rs].w;
            }
            if (!put_gradient<DT>(a, sh, ring, sl, q, token, x, false, cur)) return false;
        }
        if (kind == kEnd) return true;
        if (kind == kRow) ++rows;
        __syncwarp();
        if (lane == 0) arrive(&sh.item_empty[slot]);
    }
}

// What a CTA starts with: its barriers, and all CTAs of its cluster running.
__device__ __forceinline__ void set_up(const TokenArgs& a, Shared& sh, bool finish) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&sh.item_full[i], 1);
            mbar_init(&sh.item_empty[i], kWarps + finish);
            mbar_init(&sh.row_ready[i], 1);
        }
        for (int i = 0; i < a.ring; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], kWarps);
        }
        for (int i = 0; i < kSlots; ++i) mbar_init(&sh.shares[i], 1);
        mbar_init(&sh.next, 1);
        mbar_init(&sh.next_free, a.split);
        mbar_init_fence();
        mbar_expect_tx(&sh.next, 16);
    }
    __syncthreads();
    if (a.split > 1) cg::this_cluster().sync();
}

template <int DT, bool SUMS, bool GRAD>
__global__ void __launch_bounds__(kBlock, Shape<SUMS, GRAD>::ctas) token_kernel(const TokenArgs a) {
    extern __shared__ __align__(128) unsigned char s_raw[];
    asm volatile("griddepcontrol.launch_dependents;");
    Shared& sh = *reinterpret_cast<Shared*>(s_raw);
    unsigned char* ring = s_raw + ring_offset();
    const int t = threadIdx.x, rank = (int)(blockIdx.x % a.split);
    set_up(a, sh, SUMS || a.paired);
    wait_prior();
    bool ok = true;
    if (t < kThreads) {
        ok = work_rows<DT, SUMS, GRAD>(a, sh, ring, rank);
    } else if (t < kThreads + 32) {
        if (SUMS)
            ok = finish_rows<GRAD>(a, sh, rank);
        else if (a.paired)
            ok = find_slopes(a, sh, rank);
    } else if (t == kThreads + 32) {
        Fetcher<DT, SUMS, GRAD> f(a, sh, ring, rank);
        ok = f.ask(true) && f.run();
        if (!ok) f.drain();
    }
    if (!ok) raise_status(a.dev_status, DLM_DEV_TIMEOUT);
    __syncwarp();
    if (a.split > 1) cg::this_cluster().sync();  // no CTA ends before what others send to it has come
}

// One CTA per pair, after the sums of dlm_preference_loss: the scores, the loss, and the slope
// of every row of the pair in its state.  Bound
// by latency: three loads after each other, a sum over the CTA, the loss and a store; a
// thread's first rows are read before the sum, so that only stores follow it (8 pairs of 128
// rows: 6 us, 8 with the loads one after the other).  Every CTA reads the offsets before
// its pair's: meant for thousands of pairs, not millions.
constexpr int kPairRows = 4;
__global__ void __launch_bounds__(kThreads) pair_kernel(const TokenArgs a) {
    __shared__ double s_sum[2][kWarps];
    __shared__ int32_t s_top[kWarps];
    __shared__ float s_slope;
    asm volatile("griddepcontrol.launch_dependents;");
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int64_t i = blockIdx.x;
    wait_prior();
    // the pair's offsets, and the largest of those before them: within the rows and in order
    const int32_t given[3] = {a.offsets[2 * i], a.offsets[2 * i + 1], a.offsets[2 * i + 2]};
    int32_t top = 0;
    for (int64_t k = t; k < 2 * i; k += kThreads) top = max(top, a.offsets[k]);
    top = __reduce_max_sync(DLM_FULL_MASK, top);
    if (lane == 0) s_top[warp] = top;
    __syncthreads();
    int64_t at[3];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = max(top, s_top[w]);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        top = max(top, given[k]);
        at[k] = min((int64_t)top, a.n_rows);
        if (t == 0 && at[k] != given[k]) raise_status(a.dev_status, DLM_DEV_BAD_INDEX);
    }
    double sum[2] = {0.0, 0.0};
    float weight[kPairRows];
    bool has[kPairRows];
#pragma unroll
    for (int k = 0; k < kPairRows; ++k) {
        const int64_t r = at[0] + t + k * kThreads;
        has[k] = false;
        if (r < at[2]) {
            const float* s = a.state + r * DLM_TOKEN_STATE;
            weight[k] = a.weights ? a.weights[r] : 1.f;
            has[k] = s[1] != 0.f;  // (0: no loss of its own)
            const double term = *reinterpret_cast<const double*>(s + 4);
            sum[r >= at[1]] += term;
        }
    }
    for (int64_t r = at[0] + t + kPairRows * kThreads; r < at[2]; r += kThreads)
        sum[r >= at[1]] += *reinterpret_cast<const double*>(a.state + r * DLM_TOKEN_STATE + 4);
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        sum[0] += __shfl_xor_sync(DLM_FULL_MASK, sum[0], o);
        sum[1] += __shfl_xor_sync(DLM_FULL_MASK, sum[1], o);
    }
    if (lane == 0) {
        s_sum[0][warp] = sum[0];
        s_sum[1][warp] = sum[1];
    }
    __syncthreads();
    if (t == 0) {
        double score[2] = {0.0, 0.0};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            score[0] += s_sum[0][w];
            score[1] += s_sum[1][w];
        }
        s_slope = finish_pair(a, i, score[0], score[1]);
    }
    __syncthreads();
    const float slope = s_slope;
    auto put = [&](int64_t r, float w) {
        float* s = a.state + r * DLM_TOKEN_STATE;
        s[3] = (r >= at[1] ? -slope : slope) * w;
        s[6] = __int_as_float((int)i);
    };
#pragma unroll
    for (int k = 0; k < kPairRows; ++k)
        if (has[k]) put(at[0] + t + k * kThreads, weight[k]);
    for (int64_t r = at[0] + t + kPairRows * kThreads; r < at[2]; r += kThreads)
        if (a.state[r * DLM_TOKEN_STATE + 1] != 0.f) put(r, a.weights ? a.weights[r] : 1.f);
}

}  // namespace

// A step's workspace: the rows' state and the offsets put right.
size_t preference_workspace(int64_t n_rows, int64_t n_pairs) {
    return (size_t)n_rows * DLM_TOKEN_STATE * 4 + ((size_t)n_pairs * 2 + 1 + 3) / 4 * 16;
}

namespace {

template <typename F>
cudaError_t launch_grid(F kernel, const TokenArgs& a, unsigned grid, int block, size_t smem, int cluster, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// CTAs per row, and whether a step's row stays in the ring between its sums and its
// gradient.
template <int DT, bool SUMS, bool GRAD>
cudaError_t launch_token_kernel(TokenArgs a, cudaStream_t st) {
    using S = Shape<SUMS, GRAD>;
    constexpr int EPV = Row<DT>::EPV;
    const int64_t nv = (a.vocab + EPV - 1) / EPV, slots = (int64_t)S::ctas * a.num_sms;
    auto slice = [&](int n) { return ((nv + n - 1) / n + 7) / 8 * 8; };
    auto chunks = [&](int n) { return (slice(n) + kChunkVecs - 1) / kChunkVecs; };
    a.ring = S::ring;
    int split = 1;
    if (GRAD) {
        // Slices that the ring holds.  A step then reads a row once (2048 rows of 152064 bf16
        // with four CTAs per row 183 us; from L2 the second time, two, 184, and one, whose
        // rows in flight L2 does not hold, 230; 512 of 126464 48, 49 and 53).  A gradient
        // alone: 1024 rows of 126464 76 us with four, 83 with one.
        while (split < 8 && chunks(split) > a.ring) split *= 2;
    } else if (a.n_rows > slots && a.n_rows < 4 * slots && a.n_rows % slots > slots / 6 && a.n_rows % slots < slots * 3 / 5) {
        // whole rows would leave the last of two to four rounds to some of the CTAs (1024 rows
        // of 126464 bf16: 50 us with two, 56 with one; 912, two rounds, 47 and 43).  A second
        // launch of the rows left over, cut finer, began too late: 1024 rows took as long.
        split = 2;
    }
    // rows too few for all SMs (76 rows of 126464 bf16: 12.4 us with two CTAs each, 14.8 with
    // one, 13.1 with eight)
    while (split < 8 && a.n_rows * split < a.num_sms && slice(split) * 16 > kLeast) split *= 2;
    a.split = split;
    a.resident = chunks(split) <= a.ring;
    // the same limit whatever the call's size: calls may run side by side
    const cudaError_t e =
        cudaFuncSetAttribute(token_kernel<DT, SUMS, GRAD>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    return launch_grid(token_kernel<DT, SUMS, GRAD>, a, (unsigned)(a.n_rows * a.split), kBlock,
                       ring_offset() + (size_t)a.ring * kChunkBytes, a.split, st);
}

template <int DT>
cudaError_t run_token(TokenArgs a, cudaStream_t st) {
    if (a.op == kTokenPreference && a.sums) {
        cudaError_t e = cudaSuccess;
        if (a.workspace) {
            a.state = static_cast<float*>(a.workspace);
            a.at = reinterpret_cast<int32_t*>(a.state + a.n_rows * DLM_TOKEN_STATE);
        }
        a.paired = a.workspace && a.n_rows;  // a step: sums, then the gradient, which adds up the pairs
        a.stay_from = a.n_rows - kStays / (a.vocab * Row<DT>::ESZ);
        if (a.n_rows) e = launch_token_kernel<DT, true, false>(a, st);
        if (e != cudaSuccess) return e;
        if (a.paired) return launch_token_kernel<DT, false, true>(a, st);
        return a.n_pairs > 0 ? launch_grid(pair_kernel, a, (unsigned)a.n_pairs, kThreads, 0, 0, st) : cudaSuccess;
    }
    if (!a.sums) return launch_token_kernel<DT, false, true>(a, st);
    if (!a.grad) return launch_token_kernel<DT, true, false>(a, st);
    return launch_token_kernel<DT, true, true>(a, st);
}

}  // namespace

cudaError_t launch_token(const TokenArgs& a, int dtype, cudaStream_t st) {
    switch (dtype) {
    case DLM_BF16: return run_token<DLM_BF16>(a, st);
    case DLM_F16: return run_token<DLM_F16>(a, st);
    default: return run_token<DLM_F32>(a, st);
    }
}

}  // namespace dlm
