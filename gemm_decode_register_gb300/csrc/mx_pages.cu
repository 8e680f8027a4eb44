// mx_pages.cu -- a pool of cache pages kept on the device: sequences forked,
// grown, cut and freed in one step (remap), the pool made dense (compact),
// and the pages' copies that come of either, sm_103a.
//
// Bookkeeping (bound: latency).  Tables of a few thousand to a million
// entries, a chain of dependent phases (tally the pages' users, decide, hand
// out pages, collect the freed ones): one launch of one cluster, whose
// hardware barrier between phases costs a fraction of a launch, instead of a
// launch per phase.  Everything a phase leaves to the next lies in L2.  The
// tallies are integer atomics and all orders (pages handed out, pages freed,
// copies) follow slot and page numbers, so results do not depend on timing.
// A page whose users stay as many needs no tally: neighbouring sequences that hold
// the same page are counted together, so the prompt of a request's beams, or
// a sequence that only grows, touches no counts.
// Tables and the pool are read more than once.  Whoever writes them meanwhile (calls
// on one pool must not overlap) gets wrong pages, but no access out of bounds:
// a page is used as an index only where it is looked at again.
//
// These kernels write lengths and tables, which other kernels of the library
// read before they wait for their predecessor; so they do not let their
// dependents start early, and fence what they wrote before they end.
//
// Copies (bound: HBM): an item is some heads of one page's half in one layer;
// blocks walk the items, 16-byte vectors, eight in flight per thread.
#include "mx_common.cuh"
#include "mx_serve.h"
#include "mx_tc.cuh"

namespace mx {

constexpr int POOL_THREADS = 1024;
constexpr int POOL_WARPS = POOL_THREADS / 32;
// CTAs of a cluster, the portable most.  (One CTA is no faster however little there
// is: a step of one sequence 10.4 us by one and 10.1 by eight, of 4 14.9 and 14.5, of 32 of 2000 tokens 19.2 and
// 15.9; a compaction of 4,000 pages 15 and 15, of 16,000 27 and 17.)
constexpr int POOL_CLUSTER = 8;
constexpr int RUN = 4;           // entries per lane of a warp's task: 128 of one table row,
constexpr int GANG = 8;          // or 16 of each of eight neighbouring rows
constexpr int NO_ENTRY = -0x7FFFFFFF - 1;
enum : int { DEVERR_NO_PAGE = MX_DEVERR_NO_PAGE, DEVERR_BAD_SLOT = MX_DEVERR_BAD_SLOT };

// A page's tallies, zero between calls: users gained (or lost) in this step
// that do not write the page, and the first slot that does, counted from the
// last (slot s of S: S - s).  Compaction: entries, new place + 1.
struct __align__(8) PageTally {
    int users, writer;
};

// The pool's own memory (mx_page_pool.work).
struct PoolWork {
    PageTally *tally;   // [P]
    uint32_t *freed;    // [P / 32] bits, zero between calls
    int *word;          // (compaction) faults, zero between calls
    int *part;          // [2 * POOL_CLUSTER] counts of each CTA's range of pages
};

static size_t words_of(int P) { return ((size_t)P + 31) / 32; }

size_t pool_work_bytes(int P)
{
    return ((size_t)P * 8 + words_of(P) * 4 + 16 + 8 * POOL_CLUSTER + 255) / 256 * 256;
}

static PoolWork pool_work(const mx_page_pool &p)
{
    PoolWork w;
    char *m = static_cast<char *>(p.work);
    w.tally = reinterpret_cast<PageTally *>(m);
    m += (size_t)p.num_pages * 8;
    w.word = reinterpret_cast<int *>(m);
    w.part = w.word + 4;
    w.freed = reinterpret_cast<uint32_t *>(w.part + 2 * POOL_CLUSTER);
    return w;
}

// Everything before it is visible to the whole cluster after it.
__device__ __forceinline__ void cluster_phase()
{
    __threadfence();
    cluster_sync_all();
}

__device__ __forceinline__ PageTally tally_at(const PageTally *t, int page)
{
    const int2 v = __ldcg(reinterpret_cast<const int2 *>(t + page));
    return PageTally{v.x, v.y};
}

__device__ __forceinline__ int pages_of(long long tokens, int page_size)
{
    return tokens <= 0 ? 0 : (int)((tokens + page_size - 1) / page_size);
}

// Largest of the block's values.
__device__ __forceinline__ int block_max(int v, int *scratch)
{
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_max_sync(0xFFFFFFFFu, scratch[threadIdx.x & 31]);
}

// Sum of the values of the threads before this one, and of all.
__device__ __forceinline__ unsigned long long block_prefix(unsigned long long v, unsigned long long *scratch,
                                                           unsigned long long &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    unsigned long long w = scratch[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, w, o);
        if (lane >= o) w += y;
    }
    total = __shfl_sync(0xFFFFFFFFu, w, 31);
    const unsigned long long before = __shfl_sync(0xFFFFFFFFu, w, warp > 0 ? warp - 1 : 0);
    return x - v + (warp > 0 ? before : 0ull);
}

// ------------------------------------------------------------ remap

struct RemapArgs {
    RemapCall c;
    PoolWork w;
    int *err;
};

constexpr int CUT_CHILD = 1 << 16;  // children of a sequence: that keep all of it, and (upper half) a part

// A new sequence: its parent (or -1), tokens taken from it, tokens.
struct Slot {
    int parent, kept, tokens;
};

// What the CTAs of the cluster tell each other, in each one's shared memory.
struct RemapShared {
    int fault, late;     // faults of the tally, of the decision (a word of its own: another CTA may be ahead)
    int handed, copies;  // pages handed out, copies
    int smax[32];
    unsigned long long scan[32];
};

// (a 32-bit word of every CTA's shared memory)
__device__ __forceinline__ void all_ctas_or(const void *word, int bits)
{
    const uint32_t here = smem_u32(word);
    for (uint32_t r = 0; r < POOL_CLUSTER; ++r)
        asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(map_to_cta(here, r)), "r"(bits) : "memory");
}

// (the plan, of two words a slot, on an even word)
static __host__ __device__ size_t remap_plan_at(int S_in, int S_out) { return (4 * (size_t)S_in + 4 * (size_t)S_out + 1) / 2 * 2; }
static size_t remap_smem(int S_in, int S_out) { return sizeof(int) * (remap_plan_at(S_in, S_out) + 2 * (size_t)S_out); }

// The first thing a step needs is every sequence's length and every slot's
// parent: they are read once, into each CTA's shared memory.  A phase is then one
// round trip to L2 and a barrier.
__global__ void __launch_bounds__(POOL_THREADS, 1) kv_remap_kernel(const __grid_constant__ RemapArgs a)
{
    const RemapCall &c = a.c;
    const PoolWork &w = a.w;
    extern __shared__ int dyn[];
    int *children = dyn;                                        // [S_in]
    int *cuts = children + c.S_in;                              // [S_in] what a lone child that keeps a part keeps
    int *rows = cuts + c.S_in;                                  // [S_in]
    int *lens = rows + c.S_in;                                  // [S_in]
    Slot *slots = reinterpret_cast<Slot *>(lens + c.S_in);      // [S_out]
    int2 *plan = reinterpret_cast<int2 *>(dyn + remap_plan_at(c.S_in, c.S_out));  // [S_out] of CTA 0: first page handed out, copy's number + 1
    int *tails = lens + c.S_in + 3 * c.S_out;                   // [S_out] of CTA 0: page a growing slot writes in, or -1
    __shared__ RemapShared sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = threadIdx.x;
    const int rank = (int)cluster_ctarank();
    const int gw = warp * POOL_CLUSTER + rank, nw = POOL_WARPS * POOL_CLUSTER;
    const int ps = c.page_size, P = c.pool.num_pages;
    if (tid == 0) sh.fault = sh.late = 0;
    pdl_wait();
    cluster_sync_all();  // (before a CTA reports to the others)

    // ---- lengths and slots, children of each sequence, longest rows
    const int count = __ldcg(c.pool.count);
    int fault = 0, rows_in = 0, rows_out = 0;
    for (int p = tid; p < c.S_in; p += POOL_THREADS) {
        const int len = max(__ldcg(c.kv_len_in + p), 0), n = pages_of(len, ps);
        if (n > c.in_pages) fault |= DEVERR_BAD_PAGE;
        rows_in = max(rows_in, min(n, c.in_pages));
        lens[p] = len;
        children[p] = 0;
    }
    // References of number i of the pages that are handed out: zero, or the
    // stack is not in order.  CTA 0 fetches one for each thread before it is known
    // how many there will be.
    auto refs_of = [&](int page) { return (unsigned)page < (unsigned)P ? __ldcg(c.pool.refs + page) : 1; };
    const int next_page = rank == 0 && count <= P && tid < count ? __ldcg(c.pool.free_pages + (count - 1 - tid)) : -1;
    for (int s = tid; s < c.S_out; s += POOL_THREADS) {
        Slot n;
        n.parent = __ldcg(c.parent + s);
        n.kept = c.keep ? max(__ldcg(c.keep + s), 0) : 0x7FFFFFFF;
        n.tokens = c.add ? max(__ldcg(c.add + s), 0) : n.parent < 0 ? 0 : c.add_all;
        slots[s] = n;
    }
    __syncthreads();
    for (int s = tid; s < c.S_out; s += POOL_THREADS) {
        Slot n = slots[s];
        if (n.parent >= c.S_in) fault |= DEVERR_BAD_SLOT;
        if (n.parent < 0 || n.parent >= c.S_in) n.parent = -1;
        const int len = n.parent < 0 ? 0 : lens[n.parent];
        n.kept = min(n.kept, len);
        const long long tokens = (long long)n.kept + n.tokens;
        if (tokens > (long long)c.out_pages * ps || tokens > 0x7FFFFFFFll) fault |= DEVERR_BAD_PAGE;
        n.tokens = (int)min(tokens, 0x7FFFFFFFll);
        rows_out = max(rows_out, min(pages_of(n.tokens, ps), c.out_pages));
        slots[s] = n;
        if (n.parent >= 0) {
            atomicAdd(children + n.parent, n.kept == len ? 1 : CUT_CHILD);
            if (n.kept < len) cuts[n.parent] = n.kept;  // (used where there is one)
        }
    }
    rows_in = block_max(rows_in, sh.smax);
    rows_out = block_max(rows_out, sh.smax);
    const int chunks_in = (rows_in + 32 * RUN - 1) / (32 * RUN), chunks_out = (rows_out + 32 * RUN - 1) / (32 * RUN);
    // pages and, of what it leaves its child, full pages of each sequence
    for (int p = tid; p < c.S_in; p += POOL_THREADS) {
        rows[p] = min(pages_of(lens[p], ps), c.in_pages);
        cuts[p] = (children[p] == CUT_CHILD ? cuts[p] : lens[p]) / ps;
    }
    __syncthreads();

    // f(page, users, special) for the old tables' entries of this warp's tasks:
    // a lane takes one of GANG neighbouring sequences and four columns.
    // Neighbours that hold the same page (beams of one request, a common
    // prefix) count as one.  users: what the step leaves the page through these entries, the
    // children that keep the sequence beyond the page (a lone child that keeps a
    // part of it counts here, others by themselves), less the entries.
    // special: the page may have been counted by a child itself.  The first
    // task's entries stay in registers.
    const int gangs = (c.S_in + GANG - 1) / GANG, columns = (rows_in + 4 * RUN - 1) / (4 * RUN);
    int own[RUN];
    bool have_own = false;
    auto old_entries = [&](auto f) {
        for (int t = gw; t < gangs * columns; t += nw) {
            const int p = t % gangs * GANG + lane % GANG, j0 = t / gangs * (4 * RUN) + lane / GANG;
            const int n = p < c.S_in ? rows[p] : 0, full = p < c.S_in ? cuts[p] : 0, kids = p < c.S_in ? children[p] : 0;
            const int there = kids == CUT_CHILD ? 1 : kids % CUT_CHILD;
            const int32_t *row = c.table_in + (long long)p * c.in_stride;
            int page[RUN];
#pragma unroll
            for (int i = 0; i < RUN; ++i) {
                const int j = j0 + 4 * i;
                if (t == gw && have_own) page[i] = own[i];
                else page[i] = j < n ? max(__ldcg(row + j), -1) : NO_ENTRY;
            }
#pragma unroll
            for (int i = 0; i < RUN; ++i) {
                const int j = j0 + 4 * i;
                if (t == gw) own[i] = page[i];
                // runs of the same page: from a first lane up to the next's
                const int left = __shfl_up_sync(0xFFFFFFFFu, page[i], 1);
                const bool first = lane % GANG == 0 || page[i] != left;
                const unsigned firsts = __ballot_sync(0xFFFFFFFFu, first) >> lane >> 1;
                const int run = firsts ? __ffs((int)firsts) : 32 - lane;
                int users = (j < full ? there : 0) - 1;
#pragma unroll
                for (int o = 1; o < GANG; o <<= 1) {
                    const int more = __shfl_down_sync(0xFFFFFFFFu, users, o);
                    if (o < run) users += more;
                }
                const unsigned special = __ballot_sync(0xFFFFFFFFu, j == full || kids > CUT_CHILD) >> lane;
                if (first && page[i] != NO_ENTRY) f(page[i], users, (special & ((2u << (run - 1)) - 1u)) != 0u);
            }
        }
        have_own = true;
    };

    const int next_refs = refs_of(next_page);

    // ---- tally.  The partial page of each slot: CTA 0, a thread for each
    if (rank == 0)
        for (int s = tid; s < c.S_out; s += POOL_THREADS) {
            const Slot n = slots[s];
            const int full = n.kept / ps;
            int tail = -1;
            if (n.kept % ps != 0 && full < c.in_pages) {
                const int page = __ldcg(c.table_in + (long long)n.parent * c.in_stride + full);
                if ((unsigned)page < (unsigned)P) {
                    if (n.tokens > n.kept) atomicMax(&w.tally[tail = page].writer, c.S_out - s);
                    else atomicAdd(&w.tally[page].users, 1);
                }
            }
            tails[s] = tail;
        }
    old_entries([&](int page, int d, bool) {
        if ((unsigned)page >= (unsigned)P) fault |= DEVERR_BAD_PAGE;
        else if (d != 0) atomicAdd(&w.tally[page].users, d);
    });
    // full pages of those that take a part, with others of the same parent
    if (c.keep)
        for (int t = gw; t < c.S_out * chunks_in; t += nw) {
            const int s = t % c.S_out, j0 = t / c.S_out * (32 * RUN);
            const Slot n = slots[s];
            if (n.parent < 0 || n.kept == lens[n.parent] || children[n.parent] == CUT_CHILD) continue;
            const int32_t *row = c.table_in + (long long)n.parent * c.in_stride;
            const int full = min(n.kept / ps, c.in_pages);
            for (int j = j0 + lane; j < min(full, j0 + 32 * RUN); j += 32) {
                const int page = __ldcg(row + j);
                if ((unsigned)page < (unsigned)P) atomicAdd(&w.tally[page].users, 1);
            }
        }
    if (fault) all_ctas_or(&sh.fault, fault);
    cluster_phase();

    // ---- pages each slot is handed out, in slot order (CTA 0); pages left
    // without a user.  Not where a fault is known: lengths may not fit the tables.
    fault = *(volatile int *)&sh.fault;
    if (fault == 0) {
        int bad = 0;
        if (rank == 0) {
            constexpr int PER = (POOL_MAX_SLOTS + POOL_THREADS - 1) / POOL_THREADS;
            constexpr unsigned long long COPY = 1ull << 40;  // pages below, copies above
            const int per = (c.S_out + POOL_THREADS - 1) / POOL_THREADS, s0 = tid * per;
            unsigned long long need[PER], mine = 0;
            PageTally tally[PER];
            int refs[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int tail = i < per && s0 + i < c.S_out ? tails[s0 + i] : -1;
                if (tail >= 0) {
                    tally[i] = tally_at(w.tally, tail);
                    refs[i] = __ldcg(c.pool.refs + tail);
                }
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                need[i] = 0;
                if (i >= per || s0 + i >= c.S_out) continue;
                const Slot n = slots[s0 + i];
                need[i] = (unsigned)(pages_of(n.tokens, ps) - pages_of(n.kept, ps));
                // a page that only growing slots use stays with the first
                if (tails[s0 + i] >= 0 && !(refs[i] + tally[i].users == 0 && tally[i].writer == c.S_out - s0 - i))
                    need[i] += COPY + 1;
                mine += need[i];
            }
            unsigned long long total;
            unsigned long long at = block_prefix(mine, sh.scan, total);
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (i >= per || s0 + i >= c.S_out) continue;
                plan[s0 + i] = make_int2((int)(at & (COPY - 1)), need[i] >= COPY ? (int)(at / COPY) + 1 : 0);
                at += need[i];
            }
            if (tid == 0) {
                const unsigned long long n = total & (COPY - 1);
                if (count < 0 || count > P) bad |= DEVERR_BAD_PAGE;
                else if (n > (unsigned long long)count) bad |= DEVERR_NO_PAGE;
                sh.handed = (int)n;
                sh.copies = (int)(total / COPY);
            }
            if (count <= P) {
                const int n = (int)min(total & (COPY - 1), (unsigned long long)max(count, 0));
                if (tid < n && next_refs != 0) bad |= DEVERR_BAD_PAGE;
                for (int i = tid + POOL_THREADS; i < n; i += POOL_THREADS)
                    if (refs_of(__ldcg(c.pool.free_pages + (count - 1 - i))) != 0) bad |= DEVERR_BAD_PAGE;
            }
        }
        old_entries([&](int page, int d, bool) {
            if (d >= 0 || (unsigned)page >= (unsigned)P) return;
            const PageTally t = tally_at(w.tally, page);
            const int left = __ldcg(c.pool.refs + page) + t.users;
            if (left < 0) bad |= DEVERR_BAD_PAGE;  // fewer references than entries
            if (left == 0 && t.writer == 0) atomicOr(w.freed + (page >> 5), 1u << (page & 31));
        });
        if (bad) all_ctas_or(&sh.late, bad);
    }
    cluster_phase();

    // ---- all or nothing
    fault |= *(volatile int *)&sh.late;
    if (fault) {
        old_entries([&](int page, int, bool) {
            if ((unsigned)page >= (unsigned)P) return;
            w.tally[page] = PageTally{0, 0};
            w.freed[page >> 5] = 0u;
        });
        if (rank == 0) {
            for (int s = tid; s < c.S_out; s += POOL_THREADS) c.kv_len_out[s] = -1;
            if (tid == 0) {
                reinterpret_cast<int4 *>(c.copies)[0] = make_int4(0, 0, 0, 0);
                set_device_error(a.err, fault);
            }
        }
        cluster_phase();  // (no CTA leaves while another may report to it; lengths are read early)
        return;
    }
    const uint32_t plan0 = map_to_cta(smem_u32(plan), 0);
    for (int t = gw; t < c.S_out * max(chunks_out, 1); t += nw) {
        const int s = t % c.S_out, j0 = t / c.S_out * (32 * RUN);
        const Slot n = slots[s];
        const int end = pages_of(n.tokens, ps);
        if (j0 >= end && j0 > 0) continue;
        const int first = ld_cluster_s32(plan0 + 8 * s), copy = ld_cluster_s32(plan0 + 8 * s + 4);
        const int start = pages_of(n.kept, ps) - (copy != 0);
        const int32_t *from = c.table_in + (long long)max(n.parent, 0) * c.in_stride;
        int32_t *to = c.table_out + (long long)s * c.out_stride;
        int page[RUN];
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
            const int j = j0 + 32 * i + lane;
            const int place = count - 1 - first - (j - start);
            if (j < start) page[i] = __ldcg(from + j);
            else if (j < end) page[i] = (unsigned)place < (unsigned)P ? __ldcg(c.pool.free_pages + place) : -1;
        }
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
            const int j = j0 + 32 * i + lane;
            if (j >= end) continue;
            to[j] = page[i];
            if (j < start) continue;
            if ((unsigned)page[i] < (unsigned)P) c.pool.refs[page[i]] = 1;
            if (j == start && copy != 0)
                reinterpret_cast<int4 *>(c.copies)[copy] = make_int4(__ldcg(from + j), page[i], n.kept % ps, 0);
        }
        if (j0 == 0 && lane == 0) c.kv_len_out[s] = n.tokens;
    }
    old_entries([&](int page, int d, bool special) {
        if ((d == 0 && !special) || (unsigned)page >= (unsigned)P) return;
        // whoever comes first takes the tally
        const int refs = __ldcg(c.pool.refs + page);
        const unsigned long long v = atomicExch(reinterpret_cast<unsigned long long *>(w.tally + page), 0ull);
        if (v == 0ull) return;
        const int left = refs + (int)(uint32_t)v;
        c.pool.refs[page] = left == 0 && (v >> 32) != 0 ? 1 : left;
    });
    cluster_phase();

    // ---- the freed pages go on the stack, in page order (CTA 0)
    if (rank != 0) return;
    const int words = (P + 31) / 32;
    int top = count - sh.handed;
    for (int i0 = 0; i0 < words; i0 += POOL_THREADS) {
        const int i = i0 + tid;
        uint32_t bits = i < words ? __ldcg(w.freed + i) : 0u;
        if (__syncthreads_or(bits != 0u) == 0) continue;
        unsigned long long total;
        int at = top + (int)block_prefix((unsigned)__popc(bits), sh.scan, total);
        if (bits) w.freed[i] = 0u;
        for (; bits && at < P; bits &= bits - 1) c.pool.free_pages[at++] = 32 * i + __ffs((int)bits) - 1;
        top += (int)total;
    }
    if (tid == 0) {
        // (the stack said so of pages in use.  Found here and not before anything is written, which
        // would take a round trip to L2 more, 1 us of a step's 15)
        if (top > P) set_device_error(a.err, DEVERR_BAD_PAGE);
        *c.pool.count = min(top, P);
        reinterpret_cast<int4 *>(c.copies)[0] = make_int4(sh.copies, 0, 0, 0);
    }
}

// ------------------------------------------------------------ compact

struct CompactArgs {
    mx_page_pool pool;
    PoolWork w;
    int page_size;
    int32_t *table;
    int stride, pages, S;
    const int32_t *kv_len;
    int32_t *copies;
    int *err;
};

// U pages are in use.  The i-th free page below U takes the place of the i-th
// page in use from U on whose references are all entries of this table.
__global__ void __launch_bounds__(POOL_THREADS, 1) kv_compact_kernel(const __grid_constant__ CompactArgs a)
{
    const PoolWork &w = a.w;
    __shared__ int smax[32];
    __shared__ unsigned long long scan[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = (int)cluster_ctarank();
    const int gw = warp * POOL_CLUSTER + rank, nw = POOL_WARPS * POOL_CLUSTER;
    const int ps = a.page_size, P = a.pool.num_pages;
    // this warp's range of pages
    const int span = ((P + nw - 1) / nw + 31) / 32 * 32;
    const int lo = (int)min((long long)(rank * POOL_WARPS + warp) * span, (long long)P);
    const int hi = (int)min((long long)lo + span, (long long)P);
    pdl_wait();

    int rows = 0, fault = 0;
    for (int s = threadIdx.x; s < a.S; s += POOL_THREADS) {
        const int n = pages_of(__ldcg(a.kv_len + s), ps);
        if (n > a.pages) fault |= DEVERR_BAD_PAGE;
        rows = max(rows, min(n, a.pages));
    }
    rows = block_max(rows, smax);
    const int chunks = (rows + 32 * RUN - 1) / (32 * RUN);
    auto entries = [&](auto f) {
        for (int t = gw; t < a.S * chunks; t += nw) {
            const int s = t % a.S, j0 = t / a.S * (32 * RUN);
            const int n = min(pages_of(__ldcg(a.kv_len + s), ps), a.pages);
            int32_t *row = a.table + (long long)s * a.stride;
            int page[RUN];
#pragma unroll
            for (int i = 0; i < RUN; ++i) {
                const int j = j0 + 32 * i + lane;
                page[i] = j < n ? __ldcg(row + j) : -1;
            }
#pragma unroll
            for (int i = 0; i < RUN; ++i)
                if (j0 + 32 * i + lane < n) f(row + j0 + 32 * i + lane, page[i]);
        }
    };
    // Sum over the pages of this CTA before this warp's range and over all the
    // CTA's, of up to two counts (the second 2^32 up).
    auto range_sum = [&](unsigned long long mine, unsigned long long &total) {
        return block_prefix(lane == 0 ? mine : 0ull, scan, total);
    };
    // the CTAs' totals: of those before this one, and of all
    auto totals = [&](int slot, int &all) {
        int before = 0;
        all = 0;
        for (int r = 0; r < POOL_CLUSTER; ++r) {
            const int v = __ldcg(w.part + slot * POOL_CLUSTER + r);
            if (r < rank) before += v;
            all += v;
        }
        return before;
    };

    // ---- entries of each page; pages in use
    entries([&](int32_t *, int page) {
        if ((unsigned)page >= (unsigned)P) fault |= DEVERR_BAD_PAGE;
        else atomicAdd(&w.tally[page].users, 1);
    });
    unsigned used = 0;
    for (int p = lo + lane; p < hi; p += 32) used += __ldcg(a.pool.refs + p) > 0;
    used = __reduce_add_sync(0xFFFFFFFFu, used);
    unsigned long long total;
    range_sum(used, total);
    if (threadIdx.x == 0) w.part[rank] = (int)total;
    if (fault) atomicOr(w.word, fault);
    cluster_phase();
    auto give_up = [&](int why) {
        for (int p = lo + lane; p < hi; p += 32) w.tally[p] = PageTally{0, 0};
        if (rank == 0 && threadIdx.x == 0) {
            reinterpret_cast<int4 *>(a.copies)[0] = make_int4(0, 0, 0, 0);
            set_device_error(a.err, why);
        }
        cluster_phase();
        if (rank == 0 && threadIdx.x == 0) w.word[0] = 0;
    };
    fault = __ldcg(w.word);
    if (fault) return give_up(fault);
    int U;
    totals(0, U);
    cluster_phase();  // (the counts' places are used again)

    // ---- free places below U, pages to move from U on
    auto kind = [&](int p) {  // 1: a free place, 2: a page to move; -1: it has more entries than references
        const int r = __ldcg(a.pool.refs + p), users = tally_at(w.tally, p).users;
        if (users > max(r, 0)) return -1;
        if (p < U) return r == 0 ? 1 : 0;
        return r > 0 && users == r ? 2 : 0;
    };
    unsigned holes = 0, movers = 0;
    for (int p0 = lo; p0 < hi; p0 += 32) {
        const int k = p0 + lane < hi ? kind(p0 + lane) : 0;
        holes += __popc(__ballot_sync(0xFFFFFFFFu, k == 1));
        movers += __popc(__ballot_sync(0xFFFFFFFFu, k == 2));
        if (k < 0) fault = DEVERR_BAD_PAGE;
    }
    if (fault) atomicOr(w.word, fault);
    const unsigned long long at = __shfl_sync(0xFFFFFFFFu, range_sum(holes | ((unsigned long long)movers << 32), total), 0);
    if (threadIdx.x == 0) {
        w.part[rank] = (int)(uint32_t)total;
        w.part[POOL_CLUSTER + rank] = (int)(total >> 32);
    }
    cluster_phase();
    fault = __ldcg(w.word);
    if (fault) return give_up(fault);
    int all_holes, all_movers;
    int hole = totals(0, all_holes) + (int)(uint32_t)at, mover = totals(1, all_movers) + (int)(at >> 32);
    const int n = min(min(all_holes, all_movers), P / 2);  // (P / 2: what the list holds)
    for (int p0 = lo; p0 < hi; p0 += 32) {
        const int k = p0 + lane < hi ? kind(p0 + lane) : 0;
        const unsigned h = __ballot_sync(0xFFFFFFFFu, k == 1), m = __ballot_sync(0xFFFFFFFFu, k == 2);
        const unsigned below = (1u << lane) - 1u;
        const int i = k == 1 ? hole + __popc(h & below) : mover + __popc(m & below);
        if (k > 0 && i < n) a.copies[4 * (size_t)(1 + i) + (k == 1 ? 1 : 0)] = p0 + lane;
        hole += __popc(h);
        mover += __popc(m);
    }
    cluster_phase();

    // ---- the moves
    for (int i = gw * 32 + lane; i < n; i += nw * 32) {
        int4 *row = reinterpret_cast<int4 *>(a.copies) + 1 + i;
        const int2 v = __ldcg(reinterpret_cast<const int2 *>(row));
        if ((unsigned)v.x >= (unsigned)P || (unsigned)v.y >= (unsigned)P) continue;
        *row = make_int4(v.x, v.y, ps, 0);
        w.tally[v.x].writer = v.y + 1;
        a.pool.refs[v.y] = __ldcg(a.pool.refs + v.x);
        a.pool.refs[v.x] = 0;
    }
    cluster_phase();
    entries([&](int32_t *e, int page) {
        const int to = (unsigned)page < (unsigned)P ? tally_at(w.tally, page).writer : 0;
        if (to > 0) *e = to - 1;
    });
    unsigned empty = 0;
    for (int p = lo + lane; p < hi; p += 32) empty += __ldcg(a.pool.refs + p) == 0;
    empty = __reduce_add_sync(0xFFFFFFFFu, empty);
    const int mine = (int)__shfl_sync(0xFFFFFFFFu, range_sum(empty, total), 0);
    if (threadIdx.x == 0) w.part[rank] = (int)total;
    cluster_phase();

    // ---- the stack: the lowest page is taken first
    int all;
    int below = totals(0, all) + mine;
    for (int p0 = lo; p0 < hi; p0 += 32) {
        const int p = p0 + lane;
        const bool e = p < hi && __ldcg(a.pool.refs + p) == 0;
        const unsigned m = __ballot_sync(0xFFFFFFFFu, e);
        const int place = all - 1 - (below + __popc(m & ((1u << lane) - 1u)));
        if (e && (unsigned)place < (unsigned)P) a.pool.free_pages[place] = p;
        if (p < hi) w.tally[p] = PageTally{0, 0};
        below += __popc(m);
    }
    if (rank == 0 && threadIdx.x == 0) {
        *a.pool.count = all;
        reinterpret_cast<int4 *>(a.copies)[0] = make_int4(n, 0, 0, 0);
    }
}

// ------------------------------------------------------------ copies

constexpr int COPY_THREADS = 256;

// What is copied of a page in one half of the cache: rows (head, token) of
// `row` bytes.  Data moves in 16-byte units (the cache's base and strides are
// multiples of 16 bytes, a row is), scales in `scale_unit`s.
struct CopyPart {
    long long page_stride, head_stride, token_stride;  // bytes
    int row;                                           // bytes
};

template <int LAYERS>
struct CopyArgs {
    uint8_t *data[LAYERS][2], *scales[LAYERS][2];
    CopyPart d, s;  // s.row = 0: no scales
    int scale_unit;  // bytes: 16, 8, 4, 2 or 1
    const int4 *copies;
    int max_copies, layers, num_pages, page_size, heads, group;  // group: heads of an item
    int *err;
};

template <typename V, unsigned F>
__device__ __forceinline__ void copy_rows(const uint8_t *src, uint8_t *dst, const CopyPart &p, int heads, int tokens)
{
    // tokens that lie together make one row of each head
    const bool together = p.token_stride == p.row;
    const unsigned per_row = (unsigned)(p.row / (int)sizeof(V)) * (together ? (unsigned)tokens : 1u);
    const unsigned rows = together ? 1u : (unsigned)tokens;  // of a head
    const unsigned n = per_row * rows * (unsigned)heads;
    auto place = [&](unsigned i) {
        const unsigned r = i / per_row, col = i - r * per_row, h = together ? r : r / rows, t = together ? 0u : r - h * rows;
        return (long long)h * p.head_stride + (long long)t * p.token_stride + (long long)col * (int)sizeof(V);
    };
    // (addresses are worked out again for the stores: kept, they would cost
    // more registers than the data)
    for (unsigned i0 = threadIdx.x; i0 < n; i0 += F * COPY_THREADS) {
        V v[F];
#pragma unroll
        for (unsigned f = 0; f < F; ++f)
            if (i0 + f * COPY_THREADS < n) v[f] = __ldcs(reinterpret_cast<const V *>(src + place(i0 + f * COPY_THREADS)));
#pragma unroll
        for (unsigned f = 0; f < F; ++f)
            if (i0 + f * COPY_THREADS < n) *reinterpret_cast<V *>(dst + place(i0 + f * COPY_THREADS)) = v[f];
    }
}

__device__ __forceinline__ void copy_scales(const uint8_t *s, uint8_t *d, const CopyPart &p, int unit, int heads, int tokens)
{
    switch (unit) {
    case 16: copy_rows<uint4, 1>(s, d, p, heads, tokens); break;
    case 8: copy_rows<uint2, 1>(s, d, p, heads, tokens); break;
    case 4: copy_rows<uint32_t, 2>(s, d, p, heads, tokens); break;
    case 2: copy_rows<uint16_t, 2>(s, d, p, heads, tokens); break;
    default: copy_rows<uint8_t, 2>(s, d, p, heads, tokens); break;
    }
}

template <int LAYERS>
__global__ void __launch_bounds__(COPY_THREADS, 4) kv_copy_kernel(const __grid_constant__ CopyArgs<LAYERS> a)
{
    pdl_wait();
    // (not before: what precedes may have written the tables that the next
    // kernels read before they wait)
    pdl_trigger();
    const int n = min(max(__ldcg(&a.copies->x), 0), a.max_copies);
    const int groups = (a.heads + a.group - 1) / a.group;
    const long long items = (long long)n * a.layers * 2 * groups;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int g = (int)(it % groups);
        const long long r = it / groups;
        const int half = (int)(r & 1), layer = (int)((r >> 1) % a.layers), i = (int)((r >> 1) / a.layers);
        const int4 c = __ldcg(a.copies + 1 + i);
        const int tokens = min(c.z, a.page_size);
        if ((unsigned)c.x >= (unsigned)a.num_pages || (unsigned)c.y >= (unsigned)a.num_pages) {
            if (threadIdx.x == 0) set_device_error(a.err, DEVERR_BAD_PAGE);
            continue;
        }
        if (tokens <= 0 || c.x == c.y) continue;
        const int head = g * a.group, heads = min(a.group, a.heads - head);
        {
            uint8_t *base = a.data[layer][half] + head * a.d.head_stride;
            copy_rows<uint4, 8>(base + c.x * a.d.page_stride, base + c.y * a.d.page_stride, a.d, heads, tokens);
        }
        if (a.s.row > 0) {
            uint8_t *base = a.scales[layer][half] + head * a.s.head_stride;
            copy_scales(base + c.x * a.s.page_stride, base + c.y * a.s.page_stride, a.s, a.scale_unit, heads, tokens);
        }
    }
}

// ------------------------------------------------------------ host

cudaError_t launch_kv_remap(const DeviceState &ds, cudaStream_t st, const RemapCall &c)
{
    RemapArgs a;
    a.c = c;
    a.w = pool_work(c.pool);
    a.err = ds.err;
    const size_t smem = remap_smem(c.S_in, c.S_out);
    static unsigned char done[64];
    const cudaError_t e = allow_smem(ds, kv_remap_kernel, (int)remap_smem(POOL_MAX_SLOTS, POOL_MAX_SLOTS), done);
    if (e != cudaSuccess) return e;
    return launch_cluster_k(kv_remap_kernel, POOL_CLUSTER, dim3(POOL_CLUSTER), dim3(POOL_THREADS), smem, st, a);
}

cudaError_t launch_kv_compact(const DeviceState &ds, cudaStream_t st, const mx_page_pool &pool, int page_size,
                              int32_t *table, int stride, int pages, const int32_t *kv_len, int S, int32_t *copies)
{
    CompactArgs a;
    a.pool = pool;
    a.w = pool_work(pool);
    a.page_size = page_size;
    a.table = table;
    a.stride = stride;
    a.pages = pages;
    a.S = S;
    a.kv_len = kv_len;
    a.copies = copies;
    a.err = ds.err;
    return launch_cluster_k(kv_compact_kernel, POOL_CLUSTER, dim3(POOL_CLUSTER), dim3(POOL_THREADS), 0, st, a);
}

// Widest unit that every address of a part is a multiple of.
static int copy_unit(long long bits)
{
    return bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : bits % 2 == 0 ? 2 : 1;
}

template <int LAYERS>
static cudaError_t run_copy(const DeviceState &ds, cudaStream_t st, const mx_paged_kv *kv, int layers,
                            const int32_t *copies, int max_copies)
{
    const bool mx8 = kv->kv_fmt == MX_KV_MXFP8;
    const long long e = mx8 ? 1 : 2;
    CopyArgs<LAYERS> a;
    long long bits = 0;
    for (int l = 0; l < layers; ++l) {
        a.data[l][0] = static_cast<uint8_t *>(kv[l].k);
        a.data[l][1] = static_cast<uint8_t *>(kv[l].v);
        a.scales[l][0] = static_cast<uint8_t *>(kv[l].k_scales);
        a.scales[l][1] = static_cast<uint8_t *>(kv[l].v_scales);
        if (mx8)
            for (int h = 0; h < 2; ++h) bits |= (long long)reinterpret_cast<uintptr_t>(a.scales[l][h]);
    }
    a.d.page_stride = kv->page_stride * e;
    a.d.head_stride = kv->head_stride * e;
    a.d.token_stride = kv->token_stride * e;
    a.d.row = (int)(kv->D * e);
    a.s.page_stride = kv->scale_page_stride;
    a.s.head_stride = kv->scale_head_stride;
    a.s.token_stride = kv->scale_token_stride;
    a.s.row = mx8 ? kv->D / 32 : 0;
    a.scale_unit = copy_unit(bits | a.s.page_stride | a.s.head_stride | a.s.token_stride | a.s.row);
    a.copies = reinterpret_cast<const int4 *>(copies);
    a.max_copies = max_copies;
    a.layers = layers;
    a.num_pages = kv->num_pages;
    a.page_size = kv->page_size;
    a.heads = kv->Hkv;
    // about 32 KB an item: two rounds of a block's loads
    const long long head = (long long)kv->page_size * a.d.row;
    a.group = (int)(head >= 32768 ? 1 : 32768 / head < kv->Hkv ? 32768 / head : kv->Hkv);
    a.err = ds.err;
    const long long items = (long long)max_copies * layers * 2 * ((kv->Hkv + a.group - 1) / a.group);
    const long long most = 8ll * ds.num_sms;
    return launch_k(kv_copy_kernel<LAYERS>, dim3((unsigned)(items < most ? items : most)), dim3(COPY_THREADS), 0, st, a);
}

cudaError_t launch_kv_copy_pages(const DeviceState &ds, cudaStream_t st, const mx_paged_kv *kv, int layers,
                                 const int32_t *copies, int max_copies)
{
    if (layers <= 8) return run_copy<8>(ds, st, kv, layers, copies, max_copies);
    return run_copy<COPY_MAX_LAYERS>(ds, st, kv, layers, copies, max_copies);
}

}  // namespace mx
