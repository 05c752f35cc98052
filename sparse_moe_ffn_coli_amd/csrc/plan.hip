// plan.hip -- a serving step's plan over the paged key-value cache: from the
// lengths that the sequences have and want, the pages that go back to the
// ring of free pages and come from it, the page tables, and every new token's
// place and position.
//
// Three prefix sums over the sequences (pages returned, pages taken, tokens)
// say where each sequence's share of the ring, of the table's new entries and
// of the step's rows lies; the shares are then written flat, an entry a
// thread, whose owner is found by halving over the sums in LDS.  What bounds
// it is the chain of dependent reads (lengths, sums, ring, slots), so one
// workgroup does all of it and nothing is synchronised across workgroups; the
// rows and new table entries of large steps, which are most of the bytes, are
// left to a second launch of many workgroups, which finds the sums again from
// the first one's outputs.
#include "device_common.h"
#include "kernels.h"

namespace coli {

constexpr int PL_NT = 1024;
constexpr int PL_ROWS_NT = 256;
constexpr int PL_EACH = 4;               // rows of a thread in the second launch
constexpr int PL_STARTS = 4096;          // sequences whose sums its LDS holds (of more the first launch writes the tables)
// Rows that the first launch writes itself (one workgroup, 12 bytes a row and
// a halving over the sums: 10351 rows 16 us, 11.5 in two launches).
constexpr int PL_ONE_LAUNCH = 4096;

// Sums saturate at 2^31 - 1, past every ring (2^30 pages) and step (2^25
// rows): what lies behind such a sum is refused.
constexpr uint32_t PL_MOST = 0x7fffffffu;
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, PL_MOST); }

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t sat_step(uint32_t v)
{
    return sat_add(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false));
}

// Inclusive saturating sum over a wave.
__device__ __forceinline__ uint32_t sat_scan(uint32_t v)
{
    v = sat_step<0x111, 0xf>(v);                             // lanes 1, 2, 4, 8 below in each row of 16
    v = sat_step<0x112, 0xf>(v);
    v = sat_step<0x114, 0xf>(v);
    v = sat_step<0x118, 0xf>(v);
    v = sat_step<0x142, 0xa>(v);                             // lane 15's to rows 1 and 3, lane 31's to rows 2 and 3
    return sat_step<0x143, 0xc>(v);
}

// Inclusive sums of N values over the workgroup and their totals.  One barrier;
// ws is not read again before the next one.
template <int N>
__device__ __forceinline__ void block_sums(uint32_t (&v)[N], uint32_t (&total)[N], uint32_t (*ws)[PL_NT / 64])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = sat_scan(v[i]);
        if (lane == 63) ws[i][wave] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t w = sat_scan(lane < PL_NT / 64 ? ws[i][lane] : 0u);
        total[i] = __builtin_amdgcn_readlane(w, 63);
        const uint32_t before = __builtin_amdgcn_readlane(w, max(wave - 1, 0));
        if (wave > 0) v[i] = sat_add(v[i], before);
    }
}

// The first of n ascending inclusive sums that is larger than i (one is).
__device__ __forceinline__ int sum_owner(const uint32_t *sums, int n, uint32_t i)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] > i) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

struct PlanSeq {
    int n, t, held, need, from;          // lengths, pages, first page that may go back
    bool below;                          // would grow, but holds fewer pages than it shares: stays as it is
};

__device__ __forceinline__ PlanSeq plan_seq(const PlanLaunch &a, int b)
{
    PlanSeq s{};
    if (b >= a.B) return s;
    const int page = 1 << a.page_shift;
    s.n = min(max(a.lens[b], 0), a.cap);
    s.t = min(max(a.want[b], 0), a.cap);
    s.held = (s.n + page - 1) >> a.page_shift;
    s.need = (s.t + page - 1) >> a.page_shift;
    const int shared = a.shared ? a.shared[b] : 0;
    // New pages in the columns of shared ones would never go back, and those would be lost to the sequence.
    s.below = s.t > s.n && s.held < shared;
    if (s.below) s.t = s.n, s.need = s.held;
    s.from = min(max(s.need, shared), s.held);
    return s;
}

// In place (new_lens = lens, new_state = state) is safe: the state is read by
// everyone before the first barrier and written behind the last, a length by
// the thread that writes it.
__global__ __launch_bounds__(PL_NT) void kv_plan_kernel(PlanLaunch a, bool rows_too, bool table_too)
{
    __shared__ uint32_t ws[3][3][PL_NT / 64];
    __shared__ uint32_t sum_a[PL_NT], sum_b[PL_NT];          // inclusive sums of the chunk's sequences
    __shared__ int at_a[PL_NT], at_b[PL_NT];                 // first page of a share; length before it
    __shared__ uint32_t granted[2];                          // pages and tokens before the first refused sequence
    __shared__ int n_refused;
    const int tid = threadIdx.x;
    const uint32_t N = (uint32_t)a.n_pages;
    const uint32_t head = min((uint32_t)max(a.state[0], 0), N - 1);
    const uint32_t count = min((uint32_t)max(a.state[1], 0), N);
    auto wrap = [&](uint32_t i) { return i >= N ? i - N : i; };   // i < 2 N
    if (tid == 0) {
        granted[0] = granted[1] = PL_MOST;
        n_refused = 0;
    }

    // ---- pages that go back, to the ring's tail ----
    const int chunks = (a.B + PL_NT - 1) / PL_NT;
    if (chunks == 0) __syncthreads();                        // (else the sums' barrier)
    uint32_t back = 0;
    const uint32_t room = N - count;                         // (pages that are no one else's always fit)
    PlanSeq s{};
    for (int c = 0; c < chunks; ++c) {
        const int b0 = c * PL_NT;
        s = plan_seq(a, b0 + tid);
        uint32_t v[1] = {(uint32_t)(s.held > s.need ? s.held - s.from : 0)}, total[1];
        block_sums<1>(v, total, ws[c & 1]);
        if (total[0]) {
            sum_a[tid] = v[0];
            at_a[tid] = s.held;
            __syncthreads();
            for (uint32_t i = tid; i < min(total[0], room - back); i += PL_NT) {
                const int x = sum_owner(sum_a, PL_NT, i);
                // the last page of a share is the last one held
                const int col = at_a[x] - (int)(sum_a[x] - i);
                a.ring[wrap(wrap(head + count) + back + i)] = a.table[(size_t)(b0 + x) * a.max_pages + col];
            }
            __syncthreads();
        }
        back = min(sat_add(back, total[0]), room);
    }

    // ---- pages and rows of the sequences that grow, first come first served ----
    const uint32_t avail = count + back;
    uint32_t pages = 0, tokens = 0;                          // of the chunks before, refused ones among them
    for (int c = 0; c < chunks; ++c) {
        const int b0 = c * PL_NT, b = b0 + tid;
        if (chunks > 1) s = plan_seq(a, b);
        const uint32_t more = (uint32_t)max(s.need - s.held, 0), news = (uint32_t)max(s.t - s.n, 0);
        uint32_t v[2] = {more, news}, total[2];
        // (ws[2]: the first chunk's may follow the loop above without a barrier)
        block_sums<2>(v, total, ws[2]);
        const uint32_t upto_p = sat_add(pages, v[0]), upto_t = sat_add(tokens, v[1]);
        const bool refused = news > 0 && (upto_p > avail || upto_t > (uint32_t)a.rows);
        sum_a[tid] = v[0];
        sum_b[tid] = v[1];
        at_a[tid] = s.held;
        at_b[tid] = s.n;
        // the first refused one is the one with the smallest sums before it
        if (refused) {
            atomicMin(&granted[0], upto_p - more);
            atomicMin(&granted[1], upto_t - news);
        }
        const uint64_t who = __ballot(refused || s.below);
        if ((tid & 63) == 0 && who) atomicAdd(&n_refused, (int)__popcll(who));
        __syncthreads();
        const uint32_t end_p = min(sat_add(pages, total[0]), granted[0]), end_t = min(sat_add(tokens, total[1]), granted[1]);
        if (b < a.B) {
            a.new_lens[b] = refused ? s.n : s.t;
            a.start[b] = (int)min(upto_t - news, granted[1]);
        }
        // The table's new entries.
        for (uint32_t i = pages + tid; table_too && i < end_p; i += PL_NT) {
            const int x = sum_owner(sum_a, PL_NT, i - pages);
            const uint32_t before = x ? sum_a[x - 1] : 0u;
            a.table[(size_t)(b0 + x) * a.max_pages + at_a[x] + (int)(i - pages - before)] = a.ring[wrap(head + i)];
        }
        // The rows: a page that is new is read where it came from, so nothing waits for the table.
        if (rows_too) {
            for (uint32_t r = tokens + tid; r < end_t; r += PL_NT) {
                const int x = sum_owner(sum_b, PL_NT, r - tokens);
                const int p = at_b[x] + (int)(r - tokens - (x ? sum_b[x - 1] : 0u)), col = p >> a.page_shift;
                const int id = col < at_a[x] ? a.table[(size_t)(b0 + x) * a.max_pages + col]
                                             : a.ring[wrap(head + pages + (x ? sum_a[x - 1] : 0u) + (uint32_t)(col - at_a[x]))];
                a.slot[r] = id >= 0 && id < a.n_pages ? (id << a.page_shift) | (p & ((1 << a.page_shift) - 1)) : -1;
                a.pos[r] = p;
            }
        }
        pages = sat_add(pages, total[0]);
        tokens = sat_add(tokens, total[1]);
        __syncthreads();                                     // sums and ws are free again
    }
    const uint32_t taken = min(pages, granted[0]), live = min(tokens, granted[1]);
    if (rows_too) {
        for (uint32_t r = live + tid; r < (uint32_t)a.rows; r += PL_NT) a.slot[r] = a.pos[r] = -1;
    }
    if (tid == 0) {
        a.start[a.B] = (int)live;
        a.new_state[0] = (int)wrap(head + taken);
        a.new_state[1] = (int)(avail - taken);
        a.new_state[2] = (int)live;
        a.new_state[3] = n_refused;
    }
}

// The rows of a large step, PL_EACH a thread: the sequence of the first is
// found by halving over the starts, the next ones follow it.  A new page's
// first position is a new token's: its row writes the table's entry (TABLE;
// the pages taken before a sequence are the sum, over the sequences before, of
// what their new tokens needed more than their old lengths held).
template <bool TABLE>
__global__ __launch_bounds__(PL_ROWS_NT) void kv_plan_rows_kernel(PlanLaunch a)
{
    __shared__ int32_t starts[TABLE ? PL_STARTS + 1 : 1], taken[TABLE ? PL_STARTS + 1 : 1], ws[PL_ROWS_NT / 64];
    const int tid = threadIdx.x;
    const uint32_t N = (uint32_t)a.n_pages;
    uint32_t head = 0;
    if constexpr (TABLE) {
        int sum = 0;                                         // of the chunks before
        for (int c = 0; c < a.B; c += PL_ROWS_NT) {
            const int b = c + tid;
            int more = 0;
            if (b < a.B) {
                const int s0 = a.start[b], news = a.start[b + 1] - s0, t = a.new_lens[b];
                more = ((t + (1 << a.page_shift) - 1) >> a.page_shift) - ((t - news + (1 << a.page_shift) - 1) >> a.page_shift);
                starts[b] = s0;
            }
            const int incl = block_scan_incl<PL_ROWS_NT / 64>(more, ws) + sum;
            if (b < a.B) taken[b] = incl - more;
            sum += ws[PL_ROWS_NT / 64 - 1];
            __syncthreads();                                 // ws is free again
        }
        if (tid == 0) starts[a.B] = a.start[a.B];
        __syncthreads();
        head = (uint32_t)a.new_state[0] + (N - (uint32_t)sum);       // the ring's head before the step
        if (head >= N) head -= N;
    }
    auto start = [&](int i) { return TABLE ? starts[TABLE ? i : 0] : a.start[i]; };
    const int live = start(a.B);
    const int r0 = (blockIdx.x * PL_ROWS_NT + tid) * PL_EACH;
    if (r0 >= a.rows) return;
    int slot[PL_EACH], pos[PL_EACH];
#pragma unroll
    for (int x = 0; x < PL_EACH; ++x) slot[x] = pos[x] = -1;
    if (r0 < live) {
        int b = 0, hi = a.B;                                 // start[b] <= r0 < start[hi]
        while (hi - b > 1) {
            const int mid = (b + hi) >> 1;
            if (start(mid) <= r0) b = mid;
            else hi = mid;
        }
        int end = start(b + 1), shift = a.new_lens[b] - end; // position of row r: r + shift
        int held = 0, col = -1, id = -1;
        auto sequence = [&] {
            shift = a.new_lens[b] - end;
            held = (start(b) + shift + (1 << a.page_shift) - 1) >> a.page_shift;
            col = -1;
        };
        sequence();
#pragma unroll
        for (int x = 0; x < PL_EACH; ++x) {
            const int r = r0 + x;
            if (r >= live) break;
            if (r >= end) {
                do end = start(++b + 1);
                while (r >= end);
                sequence();
            }
            const int p = r + shift;
            int32_t *entry = a.table + (size_t)b * a.max_pages + (p >> a.page_shift);
            if ((p >> a.page_shift) != col) {
                col = p >> a.page_shift;
                if (!TABLE || col < held) {
                    id = *entry;
                } else {
                    uint32_t i = head + (uint32_t)(taken[TABLE ? b : 0] + col - held);
                    id = a.ring[i >= N ? i - N : i];
                }
            }
            if (TABLE && col >= held && (p & ((1 << a.page_shift) - 1)) == 0) *entry = id;
            pos[x] = p;
            slot[x] = id >= 0 && id < a.n_pages ? (id << a.page_shift) | (p & ((1 << a.page_shift) - 1)) : -1;
        }
    }
    if (r0 + PL_EACH <= a.rows) {
        *reinterpret_cast<int4 *>(a.slot + r0) = int4{slot[0], slot[1], slot[2], slot[3]};
        *reinterpret_cast<int4 *>(a.pos + r0) = int4{pos[0], pos[1], pos[2], pos[3]};
        return;
    }
    for (int x = 0; x < PL_EACH && r0 + x < a.rows; ++x) {
        a.slot[r0 + x] = slot[x];
        a.pos[r0 + x] = pos[x];
    }
}

hipError_t launch_kv_plan(const PlanLaunch &a, hipStream_t st)
{
    const bool one = a.rows <= PL_ONE_LAUNCH;
    const bool sums = a.B <= PL_STARTS;
    kv_plan_kernel<<<1, PL_NT, 0, st>>>(a, one, one || !sums);
    if (!one) {
        constexpr int per = PL_ROWS_NT * PL_EACH;
        const int n = (a.rows + per - 1) / per;
        if (sums) kv_plan_rows_kernel<true><<<n, PL_ROWS_NT, 0, st>>>(a);
        else kv_plan_rows_kernel<false><<<n, PL_ROWS_NT, 0, st>>>(a);
    }
    return hipGetLastError();
}

}  // namespace coli
