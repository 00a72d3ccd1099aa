// paged_plan.cu -- a serving step's plan: the pages that sequences give back and take, the block tables, and the
// rows' sequences and positions, from the sequences' lengths and new tokens.
//
//   want_b = ceil((length_b + new_b) / page_tokens);  pages held_b -> want_b;  rows start_b .. start_b + new_b - 1
//
// All of it follows from three running sums over the sequences (new tokens, pages given back, pages needed), which
// each block takes for itself, a run of sequences a thread; what is then written (rows, pages onto the stack, pages off
// it) is laid out flat over all threads, an item finding its sequence by bisection of the sums in shared memory, so that
// one long sequence and thousands of short ones spread alike.  One thread-block cluster (of one block where there is
// little): its barrier stands between the reads of what is changed in place (held, the stack, the lengths where `ends` is
// the same buffer) and the writes, and again between the pages put onto the stack and those taken off it.
//
// What it takes, of steps that take pages and steps that give them back in turn: 64 sequences of a token each 5.4 us, 1,024 sequences
// and 65,536 rows 8.9 us (by graph replay; 0.6 MB: all of it latency, dependent loads and five block barriers and two of the cluster;
// a kernel that adds to one number takes 1.3).
#include "paged.cuh"

namespace step5 {

namespace {

constexpr int64_t kFar = 1 << 30;  // past every count of rows or pages; the stored sums stop here
enum : uint8_t { kFits = 1, kNeeds = 2 };

size_t plan_smem(int B) { return (size_t)(4 * B + 3) * 4 + (size_t)B; }

// The last index i of 0 .. B with sums[i] <= x (sums ascend from 0).
__device__ __forceinline__ int owner(const int32_t* sums, int B, int x) {
    int lo = 0, hi = B + 1;  // sums[lo] <= x, and sums[hi] > x
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// The sum of x over the block's threads before this one, and (in all) over all of them.  s: a number a warp.
template <int THREADS>
__device__ __forceinline__ int64_t before(int64_t x, int64_t* s, int64_t& all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t inc = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == 31) s[warp] = inc;
    __syncthreads();
    int64_t w = lane < THREADS / 32 ? s[lane] : 0, sum = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += o;
    }
    all = __shfl_sync(0xffffffffu, sum, 31);
    return inc - x + __shfl_sync(0xffffffffu, sum - w, warp);
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) paged_plan_kernel(PlanParams p) {
    extern __shared__ int32_t smem[];
    int32_t* s_start = smem;                  // [B + 1] first row, at most N
    int32_t* s_less = s_start + p.B + 1;      // [B + 1] pages given back before the sequence
    int32_t* s_need = s_less + p.B + 1;       // [B + 1] pages needed before it
    int32_t* s_len = s_need + p.B + 1;        // [B]
    uint8_t* s_flag = reinterpret_cast<uint8_t*>(s_len + p.B);
    __shared__ int64_t s_sum[3][THREADS / 32];
    __shared__ int s_taken;
    const int tid = threadIdx.x;
    const int at = blockIdx.x * THREADS + tid, all = gridDim.x * THREADS;
    if (tid == 0) s_taken = 0;
    pdl_wait();
    pdl_launch_dependents();

    // the sequences' numbers (for now new tokens and held pages where the sums will be), then a run of sequences a thread
    int count = *p.free_count;
    for (int b = tid; b < p.B; b += THREADS) {
        s_len[b] = p.lengths[b];
        s_start[b] = p.new_tokens[b];
        s_need[b] = p.held[b];
    }
    bool bad = count < 0 || count > p.num_pages;
    count = min(max(count, 0), p.num_pages);
    __syncthreads();
    const int each = (p.B + THREADS - 1) / THREADS, b0 = min(p.B, tid * each), b1 = min(p.B, b0 + each);
    const int64_t cap = (int64_t)p.page_tokens * p.table_len;
    int64_t mine = 0, rows, less, need;
    for (int b = b0; b < b1; ++b) mine += max(s_start[b], 0);
    const int64_t start0 = before<THREADS>(mine, s_sum[0], rows);
    // pages wanted and held: a sequence out of range, or whose rows lie past N, takes part in nothing else
    auto pages_of = [&](int b, int64_t& start, int& l, int& n) {
        const int len = s_len[b], more = s_start[b], held = s_need[b];
        const bool good = len >= 0 && more >= 0 && (int64_t)len + more <= cap && held >= 0 && held <= p.table_len && start + more <= p.N;
        start += max(more, 0);
        const int want = good ? (int)(((uint32_t)len + (uint32_t)more + (uint32_t)p.page_tokens - 1u) / (uint32_t)p.page_tokens) : held;
        l = max(held - want, 0);
        n = max(want - held, 0);
        return good;
    };
    int64_t start = start0, less0 = 0, need0 = 0;
    for (int b = b0; b < b1; ++b) {
        int l, n;
        if (!pages_of(b, start, l, n)) bad = true;
        less0 += l, need0 += n;
    }
    less0 = before<THREADS>(less0, s_sum[1], less);
    need0 = before<THREADS>(need0, s_sum[2], need);
    start = start0;
    for (int b = b0; b < b1; ++b) {
        const int64_t first = start;
        int l, n;
        const bool good = pages_of(b, start, l, n);
        s_start[b] = (int)min(first, (int64_t)p.N);
        s_less[b] = (int)min(less0, kFar);
        s_need[b] = (int)min(need0, kFar);
        s_flag[b] = (good ? kFits : 0) | (n > 0 ? kNeeds : 0);
        less0 += l, need0 += n;
    }
    if (tid == 0) {
        s_start[p.B] = (int)min(rows, (int64_t)p.N);
        s_less[p.B] = (int)min(less, kFar);
        s_need[p.B] = (int)min(need, kFar);
    }
    const int back = (int)min(less, kFar);
    if (back > p.num_pages - count) bad = true;
    const int have = min(count + back, p.num_pages);
    __syncthreads();
    // what is granted: from the first sequence whose pages run out on, none that needs pages
    auto granted = [&](int b) {
        const uint8_t f = s_flag[b];
        return (f & kFits) && (!(f & kNeeds) || s_need[b + 1] <= have);
    };
    int taken = 0;
    for (int b = tid; b < p.B; b += THREADS)
        if ((s_flag[b] & kNeeds) && granted(b)) taken = max(taken, s_need[b + 1]);
    if (taken) atomicMax(&s_taken, taken);
    cluster_sync();  // (also the block's barrier) everything that is changed below has been read
    taken = s_taken;

    auto rows_of = [&](int b) { return s_start[b + 1] - s_start[b]; };  // (of a sequence that fits)
    auto want_of = [&](int b) { return (int)(((int64_t)s_len[b] + rows_of(b) + p.page_tokens - 1) / p.page_tokens); };
    for (int x = at; x < min(back, p.num_pages - count); x += all) {
        const int b = owner(s_less, p.B, x);
        const int page = p.block_table[(int64_t)b * p.table_len + want_of(b) + (x - s_less[b])];
        if (page < 0 || page >= p.num_pages) bad = true;
        p.free_pages[count + x] = page;
    }
    for (int b = at; b < p.B; b += all) {
        const bool ok = granted(b);
        const int len = s_len[b], more = ok ? rows_of(b) : 0, end = len + more;
        p.row_start[b] = s_start[b];
        p.granted[b] = more;
        p.ends[b] = end;
        p.region_begin[b] = len >= 0 ? len >> 3 : 0;
        p.region_end[b] = len >= 0 ? end >> 3 : 0;
        if (ok) p.held[b] = want_of(b);
    }
    // (a warp takes 128 rows at a time, four a lane: the next is found from the one before)
    for (int n0 = (at >> 5) * 128 + (at & 31); n0 < p.N; n0 += 4 * all) {
        int b = owner(s_start, p.B, n0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = n0 + 32 * i;
            if (n >= p.N) break;
            while (b < p.B && s_start[b + 1] <= n) ++b;
            const bool real = b < p.B && granted(b);
            p.row_seq[n] = real ? b : -1;
            p.row_pos[n] = real ? s_len[b] + (n - s_start[b]) : -1;
        }
    }
    if (back > 0 && taken > 0) cluster_sync();  // (the same for every block)
    for (int x = at; x < taken; x += all) {
        const int b = owner(s_need, p.B, x), page = p.free_pages[have - taken + x];
        if (page < 0 || page >= p.num_pages) bad = true;
        p.block_table[(int64_t)b * p.table_len + want_of(b) - (s_need[b + 1] - s_need[b]) + (x - s_need[b])] = page;
    }
    if (blockIdx.x == 0 && tid == 0) {
        p.row_start[p.B] = s_start[p.B];
        *p.free_count = have - taken;
    }
    if (bad) raise_status(p.status, kDevRange);
}

}  // namespace

namespace {
template <int THREADS>
cudaError_t launch(const PlanParams& p, unsigned ctas, cudaStream_t stream, bool pdl) {
    static std::atomic<uint64_t> attr_set{0};
    cudaError_t e = once_per_device(attr_set, [] {
        return cudaFuncSetAttribute(paged_plan_kernel<THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)plan_smem(kPlanMaxSeqs));
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = plan_smem(p.B);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, paged_plan_kernel<THREADS>, p);
}
}  // namespace

cudaError_t launch_paged_plan(const PlanParams& p, cudaStream_t stream, bool pdl) {
    // One block of 256 threads, or a cluster of 8 of 1,024 (whose barriers cost more than little work spread), microseconds of steps
    // that move no page: 64 sequences of a row each 5.0 and 5.6, of 15 rows 5.2 and 5.5, of 62 8.0 and 5.6; 256 of a row each 6.8 and
    // 7.1, 500 7.9 and 7.5, 1,000 9.5 and 8.3, 2,048 15.1 and 9.8.
    return (int64_t)p.N + p.B <= 1024 ? launch<256>(p, 1, stream, pdl) : launch<1024>(p, 8, stream, pdl);
}

}  // namespace step5
