// paged_plan.cu -- a serving step's plan: the pages that sequences give back and take, the block tables, and the
// rows' sequences and positions, from the sequences' lengths and new tokens.
//
//   want_b = ceil((length_b + new_b) / page_tokens);  pages held_b -> want_b;  rows start_b .. start_b + new_b - 1
//
// All of it follows from three running sums over the sequences (new tokens, pages given back, pages needed), which
// each block takes for itself; what is then written (rows, pages onto the stack, pages off it) is laid out flat over
// all threads, an item finding its sequence by bisection of the sums in shared memory, so that one long sequence
// and thousands of short ones spread alike.  One thread-block cluster: its barrier stands between the reads of
// what is changed in place (held, the stack, the lengths where `ends` is the same buffer) and the writes, and again
// between the pages put onto the stack and those taken off it.
#include "paged.cuh"

namespace step5 {

namespace {

constexpr int kPlanThreads = 512, kPlanWarps = kPlanThreads / 32;
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

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(PlanParams p) {
    extern __shared__ int32_t smem[];
    int32_t* s_start = smem;                  // [B + 1] first row, at most N
    int32_t* s_less = s_start + p.B + 1;      // [B + 1] pages given back before the sequence
    int32_t* s_need = s_less + p.B + 1;       // [B + 1] pages needed before it
    int32_t* s_len = s_need + p.B + 1;        // [B]
    uint8_t* s_flag = reinterpret_cast<uint8_t*>(s_len + p.B);
    __shared__ int64_t s_sum[3][kPlanWarps];
    __shared__ int s_taken;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int at = blockIdx.x * kPlanThreads + tid, all = gridDim.x * kPlanThreads;
    const bool first = blockIdx.x == 0;
    if (tid == 0) s_taken = 0;
    pdl_wait();
    pdl_launch_dependents();

    // the sums, a block of sequences at a time
    int count = *p.free_count;
    bool bad = count < 0 || count > p.num_pages;
    count = min(max(count, 0), p.num_pages);
    const int64_t cap = (int64_t)p.page_tokens * p.table_len;
    int64_t rows = 0, less = 0, need = 0;  // of the blocks before
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int64_t v[3] = {0, 0, 0};
        bool good = false;
        int want = 0, held = 0, len = 0;
        if (b < p.B) {
            len = p.lengths[b];
            const int more = p.new_tokens[b];
            held = p.held[b];
            good = len >= 0 && more >= 0 && (int64_t)len + more <= cap && held >= 0 && held <= p.table_len;
            bad |= !good;
            v[0] = max(more, 0);
            if (good) want = (int)(((int64_t)len + more + p.page_tokens - 1) / p.page_tokens);
        }
        // rows first: a sequence whose rows lie past N takes part in nothing else
        auto scan = [&](int64_t x, int which) {  // the sum before this thread's, in the block
            int64_t inc = x;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t o = __shfl_up_sync(0xffffffffu, inc, d);
                if (lane >= d) inc += o;
            }
            if (lane == 31) s_sum[which][warp] = inc;
            return inc - x;
        };
        auto total = [&](int which, int64_t& before) {
            int64_t sum = 0;
#pragma unroll
            for (int w = 0; w < kPlanWarps; ++w) {
                if (w < warp) before += s_sum[which][w];
                sum += s_sum[which][w];
            }
            return sum;
        };
        int64_t start = scan(v[0], 0) + rows;
        __syncthreads();
        const int64_t more_rows = total(0, start);
        const bool fits = good && start + v[0] <= p.N;
        if (b < p.B && good && !fits) bad = true;
        if (fits) {
            v[1] = max(held - want, 0);
            v[2] = max(want - held, 0);
        }
        int64_t l = scan(v[1], 1) + less, n = scan(v[2], 2) + need;
        __syncthreads();
        const int64_t more_less = total(1, l), more_need = total(2, n);
        if (b < p.B) {
            s_start[b] = (int)min(start, (int64_t)p.N);
            s_less[b] = (int)min(l, kFar);
            s_need[b] = (int)min(n, kFar);
            s_len[b] = len;
            s_flag[b] = (fits ? kFits : 0) | (v[2] > 0 ? kNeeds : 0);
        }
        rows += more_rows, less += more_less, need += more_need;
        __syncthreads();  // (s_sum is free again)
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
    for (int b = tid; b < p.B; b += kPlanThreads)
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
    for (int n = at; n < p.N; n += all) {
        const int b = owner(s_start, p.B, n);
        const bool real = b < p.B && granted(b);
        p.row_seq[n] = real ? b : -1;
        p.row_pos[n] = real ? s_len[b] + (n - s_start[b]) : -1;
    }
    if (back > 0 && taken > 0) cluster_sync();  // (the same for every block)
    for (int x = at; x < taken; x += all) {
        const int b = owner(s_need, p.B, x), page = p.free_pages[have - taken + x];
        if (page < 0 || page >= p.num_pages) bad = true;
        p.block_table[(int64_t)b * p.table_len + want_of(b) - (s_need[b + 1] - s_need[b]) + (x - s_need[b])] = page;
    }
    if (first && tid == 0) {
        p.row_start[p.B] = s_start[p.B];
        *p.free_count = have - taken;
    }
    if (bad) raise_status(p.status, kDevRange);
}

}  // namespace

cudaError_t launch_paged_plan(const PlanParams& p, cudaStream_t stream, bool pdl) {
    static std::atomic<uint64_t> attr_set{0};
    cudaError_t e = once_per_device(attr_set, [] {
        return cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)plan_smem(kPlanMaxSeqs));
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((int64_t)p.N + p.B <= 4 * kPlanThreads ? 1u : 8u);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = plan_smem(p.B);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cfg.gridDim.x;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, paged_plan_kernel, p);
}

}  // namespace step5
