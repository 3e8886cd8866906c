// Block tables and slot maps built on the GPU from request lengths, and the
// return of blocks: the device-resident counterpart of the host allocator.
//
// State: one reference count per block (0 = free) and the block tables.  Growing
// sequence b from start to end positions takes
//     need_b = ceil(end_b / bs) - ceil(start_b / bs)
// blocks, the lowest-numbered free ones, sequences in order ("Paged KV Cache -
// AI infra interview lesson", Walk the Shapes First: a sequence takes a block
// exactly when a position p has p % bs == 0).  With N_b = need_0 + .. + need_b
// and F free blocks, sequence b is granted its blocks iff N_b <= F or need_b is
// 0, and the r-th free block (r = 0, 1, ..) goes to the sequence with
// N_{b-1} <= r < N_b.  New position p gets slot table[b][p / bs] * bs + p % bs.
//
// What has to move: every count once (4 B per block), and 4 B per table entry,
// count and slot written; at serving sizes (80 KB of counts, a few hundred
// slots) that is far below a microsecond, so the calls are bound by launches
// and dependent loads.  Two launches: the free blocks of every chunk of
// kTabThreads counts and the prefix of the needs (one CTA) first, then the
// assignment, in which a chunk's CTA knows its blocks' ranks from the sum of
// the earlier chunks' free counts.  The CTA that takes a block writes its
// count, its table entry and the slots of its positions, so nothing waits for
// another CTA's writes and the result does not depend on their order.  (512 prompts of up
// to 4096 tokens, 262144 blocks: 16 us with the return of the blocks, of which the million
// slots are 4 MB.)  A small growth is one CTA that does both steps.
#include <cuda_runtime.h>

#include "pkv_internal.h"
#include "pkv_pdl.cuh"

namespace pkv {
namespace {

constexpr int kTabThreads = 512;
constexpr int kTabWarps = kTabThreads / 32;
constexpr int kShrinkThreads = 128;
constexpr int kMaxTabChunks = 2048;      // chunks of ref_counts (every assigning CTA sums all their free counts)
constexpr int kTabSmemSeqs = 4096;       // need prefixes kept in shared memory up to this many sequences

// Up to these sizes one CTA grows the tables alone, in one launch and without a workspace
// to allocate.  A grow and a shrink, us, one launch / two, on the GPU in a graph and from
// Python: 64 sequences by a token each, 20000 blocks: 6.2 / 7.3, 21 / 25; 1024 by up to 8,
// 32768 blocks: 9.5 / 10.9, 22 / 25.  At the limits themselves (1024 by 8) the GPU times
// tie, 12.7 / 12.1, and what is gained is a launch and an allocation on the host, 21 / 25:
// nothing in a captured step.  By 16 tokens each the one CTA takes 18.1 / 13.6 on the GPU:
// it writes the slots alone.
constexpr int kOneThreads = 1024, kOneWarps = kOneThreads / 32;
constexpr int kOneSeqs = kOneThreads;           // a thread per sequence
constexpr int kOneBlocks = 32 * kOneThreads;    // a thread keeps 32 free bits
constexpr int kOneTokens = 8 * kOneThreads;

// A sequence's growth as both kernels see it.
struct Growth {
    int64_t start, end;
    int64_t held, grown;  // blocks before and after
    bool valid;
};

__device__ __forceinline__ Growth growth_of(int32_t start, int32_t end, int32_t bs, int32_t max_blocks) {
    Growth g;
    g.start = start;
    g.end = end;
    // 32 bits hold both sums (a 64-bit division costs as much as the rest of this); negative
    // lengths are not valid
    g.held = (static_cast<uint32_t>(start) + static_cast<uint32_t>(bs) - 1) / static_cast<uint32_t>(bs);
    g.grown = (static_cast<uint32_t>(end) + static_cast<uint32_t>(bs) - 1) / static_cast<uint32_t>(bs);
    g.valid = start >= 0 && end >= start && g.grown <= max_blocks;
    return g;
}

// Inclusive scan of one value per thread over the CTA; `total` gets the sum.
template <typename V>
__device__ __forceinline__ V block_scan(V v, V *warp_sums, V &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const V up = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += up;
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    V before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kTabWarps; ++w) {
        if (w < warp) before += warp_sums[w];
        sum += warp_sums[w];
    }
    total = sum;
    __syncthreads();  // warp_sums may be reused by the caller
    return v + before;
}

// CTA 0: need_prefix[0 .. B] (saturated) and cu_new[0 .. B].  CTA 1 + c: the
// free blocks of chunk c.
__global__ void __launch_bounds__(kTabThreads)
table_count_kernel(const int32_t *__restrict__ starts, const int32_t *__restrict__ ends, int32_t B, int32_t bs,
                   int32_t max_blocks, const int32_t *__restrict__ ref_counts, int32_t num_blocks, int32_t chunk,
                   int32_t *__restrict__ need_prefix, int32_t *__restrict__ chunk_free, int32_t *__restrict__ cu_new,
                   int32_t *__restrict__ err_flag) {
    __shared__ int64_t sums[kTabWarps];
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x > 0) {
        const int64_t c0 = static_cast<int64_t>(blockIdx.x - 1) * chunk;
        const int64_t c1 = min(c0 + chunk, static_cast<int64_t>(num_blocks));
        int64_t mine = 0, total;
        for (int64_t i = c0 + threadIdx.x; i < c1; i += kTabThreads) mine += ref_counts[i] == 0;
        block_scan(mine, sums, total);
        if (threadIdx.x == 0) chunk_free[blockIdx.x - 1] = static_cast<int32_t>(total);
        return;
    }
    int64_t need_base = 0, cu_base = 0;
    bool bad = false, over = false;
    if (threadIdx.x == 0) need_prefix[0] = cu_new[0] = 0;
    for (int b0 = 0; b0 < B; b0 += kTabThreads) {
        const int b = b0 + threadIdx.x;
        int64_t need = 0, count = 0, total;
        if (b < B) {
            const Growth g = growth_of(starts[b], ends[b], bs, max_blocks);
            bad = bad || !g.valid;
            need = g.valid ? g.grown - g.held : 0;
            count = max(g.end - g.start, static_cast<int64_t>(0));
        }
        const int64_t n = need_base + block_scan(need, sums, total);
        need_base += total;
        const int64_t c = cu_base + block_scan(count, sums, total);
        cu_base += total;
        if (b < B) {
            over = over || c > INT32_MAX;
            need_prefix[b + 1] = static_cast<int32_t>(min(n, static_cast<int64_t>(INT32_MAX)));
            cu_new[b + 1] = static_cast<int32_t>(min(c, static_cast<int64_t>(INT32_MAX)));
        }
    }
    if (err_flag) {
        if (bad) atomicOr(err_flag, PKV_ERRBIT_CONTEXT);
        if (over) atomicOr(err_flag, PKV_ERRBIT_SPAN);
    }
}

// Largest i in [0, n] with prefix[i] <= v (prefix[0] = 0, non-decreasing).
__device__ __forceinline__ int last_at_most(const int32_t *prefix, int n, int32_t v) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= v) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// CTAs [0, chunks): chunk c's free blocks of rank below the granted total go to
// their sequences.  The other CTAs, one warp per sequence: the slots of the
// positions in the block held already, and the -1 of sequences that get nothing.
__global__ void __launch_bounds__(kTabThreads)
table_assign_kernel(int32_t *__restrict__ block_tables, int32_t max_blocks, const int32_t *__restrict__ starts,
                    const int32_t *__restrict__ ends, int32_t B, int32_t bs, int32_t *__restrict__ ref_counts,
                    int32_t num_blocks, int32_t chunk, int32_t chunks, const int32_t *__restrict__ need_prefix,
                    const int32_t *__restrict__ chunk_free, const int32_t *__restrict__ cu_new,
                    int32_t *__restrict__ slots, int64_t num_slots_out, int32_t *__restrict__ err_flag) {
    __shared__ int64_t sums[kTabWarps];
    __shared__ int32_t s_prefix[kTabSmemSeqs + 1];
    __shared__ int32_t e_id[kTabThreads], e_len[kTabThreads];
    __shared__ int64_t e_out[kTabThreads];
    pdl_wait();
    pdl_trigger();
    const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // free blocks before this CTA's chunk, and in all
    int64_t before = 0, all = 0;
    for (int i = threadIdx.x; i < chunks; i += kTabThreads) {
        const int32_t f = chunk_free[i];
        if (i < c) before += f;
        all += f;
    }
    int64_t base, free_total;
    block_scan(before, sums, base);
    block_scan(all, sums, free_total);
    // positions past the last new token: padding
    const int64_t tokens = cu_new[B];
    for (int64_t k = tokens + static_cast<int64_t>(c) * kTabThreads + threadIdx.x; k < num_slots_out;
         k += static_cast<int64_t>(gridDim.x) * kTabThreads)
        slots[k] = -1;

    if (c >= chunks) {
        const int b = (c - chunks) * kTabWarps + warp;
        if (b >= B) return;
        const Growth g = growth_of(starts[b], ends[b], bs, max_blocks);
        const int64_t out0 = cu_new[b];
        int32_t *row = block_tables + static_cast<int64_t>(b) * max_blocks;
        const bool granted = g.valid && (g.grown == g.held || need_prefix[b + 1] <= free_total);
        int64_t upto = g.end;  // this warp writes the slots of [start, upto)
        int32_t id = -1;
        if (granted) {
            upto = min(g.end, g.held * bs);  // the block that holds position start - 1, when it is not full
            if (upto > g.start) {
                id = row[g.start / bs];
                if (id < 0 || id >= num_blocks) {
                    id = -1;
                    if (lane == 0 && err_flag) atomicOr(err_flag, PKV_ERRBIT_BLOCK_RANGE);
                }
            }
        } else if (g.valid) {
            for (int64_t j = g.held + lane; j < g.grown; j += 32) row[j] = -1;
            if (lane == 0 && err_flag) atomicOr(err_flag, PKV_ERRBIT_NO_BLOCKS);
        }
        // as far as the slot map goes: the span of lengths that are not valid may be 2^32
        const int64_t stop = min(upto, g.start + max(num_slots_out - out0, static_cast<int64_t>(0)));
        for (int64_t p = g.start + lane; p < stop; p += 32)
            slots[out0 + p - g.start] = id < 0 ? -1 : static_cast<int32_t>(id * static_cast<int64_t>(bs) + p % bs);
        if (lane == 0 && err_flag && out0 + max(g.end - g.start, static_cast<int64_t>(0)) > num_slots_out)
            atomicOr(err_flag, PKV_ERRBIT_SPAN);
        return;
    }

    if (base >= free_total || base >= need_prefix[B]) return;  // nothing free here, or nothing left to hand out
    const int32_t *prefix = need_prefix;
    if (B <= kTabSmemSeqs) {
        for (int i = threadIdx.x; i <= B; i += kTabThreads) s_prefix[i] = need_prefix[i];
        __syncthreads();
        prefix = s_prefix;
    }
    // granted blocks: the largest prefix of the needs that the free blocks cover
    const int32_t granted = prefix[last_at_most(prefix, B, static_cast<int32_t>(free_total))];
    const int64_t c0 = static_cast<int64_t>(c) * chunk, c1 = min(c0 + chunk, static_cast<int64_t>(num_blocks));
    for (int64_t i0 = c0; i0 < c1 && base < granted; i0 += kTabThreads) {
        const int64_t i = i0 + threadIdx.x;
        const int64_t is_free = i < c1 && ref_counts[i] == 0;
        int64_t found;
        const int64_t mine = block_scan(is_free, sums, found) - 1;  // rank inside this tile
        const int64_t rank = base + mine;
        if (is_free && rank < granted) {
            const int b = last_at_most(prefix, B, static_cast<int32_t>(rank));
            const Growth g = growth_of(starts[b], ends[b], bs, max_blocks);
            const int64_t j = g.held + rank - prefix[b];  // logical block
            ref_counts[i] = 1;
            block_tables[static_cast<int64_t>(b) * max_blocks + j] = static_cast<int32_t>(i);
            e_id[mine] = static_cast<int32_t>(i);
            e_out[mine] = cu_new[b] + j * bs - g.start;  // slot map index of the block's first position
            e_len[mine] = static_cast<int32_t>(min(static_cast<int64_t>(bs), g.end - j * bs));
        }
        __syncthreads();
        // Positions of a block as far as the slot map can hold any.  taken * span <= num_blocks * bs
        // < 2^31, and one step past it is in 32 unsigned bits.
        const uint32_t taken = static_cast<uint32_t>(min(found, granted - base));
        const uint32_t span = static_cast<uint32_t>(min(static_cast<int64_t>(bs), num_slots_out));
        for (uint32_t x = threadIdx.x; x < taken * span; x += kTabThreads) {
            const int32_t e = x / span, o = x - e * span;
            const int64_t k = e_out[e] + o;
            if (o < e_len[e] && k < num_slots_out) slots[k] = e_id[e] * bs + o;
        }
        base += found;
        __syncthreads();  // the entries are read before the next tile's overwrite them
    }
}

// The whole growth by one CTA: needs and their prefix (a thread per sequence), free
// bits and their ranks (32 blocks per thread), then kOneThreads ranks at a time.
__global__ void __launch_bounds__(kOneThreads)
table_grow_one_kernel(int32_t *__restrict__ block_tables, int32_t max_blocks, const int32_t *__restrict__ starts,
                      const int32_t *__restrict__ ends, int32_t B, int32_t bs, int32_t *__restrict__ ref_counts,
                      int32_t num_blocks, int32_t *__restrict__ cu_new, int32_t *__restrict__ slots, int32_t num_slots_out,
                      int32_t *__restrict__ err_flag) {
    __shared__ int64_t w_need[kOneWarps], w_count[kOneWarps + 1];
    __shared__ int32_t w_free[kOneWarps + 1];
    __shared__ int32_t s_prefix[kOneSeqs + 1], s_cu[kOneSeqs], s_start[kOneSeqs], s_end[kOneSeqs];
    __shared__ int32_t e_id[kOneThreads], e_out[kOneThreads], e_len[kOneThreads];
    pdl_wait();
    pdl_trigger();
    const int b = threadIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // bit i: block 32 b + i is free
    uint32_t free_bits = 0;
#pragma unroll
    for (int k = 0; k < 32; ++k) {
        const int i = 1024 * warp + 32 * k + lane;
        const uint32_t word = __ballot_sync(0xffffffffu, i < num_blocks && ref_counts[i] == 0);
        if (lane == k) free_bits = word;
    }
    Growth g{};
    if (b < B) g = growth_of(starts[b], ends[b], bs, max_blocks);
    const int64_t need = b < B && g.valid ? g.grown - g.held : 0;
    const int64_t count = b < B ? max(g.end - g.start, static_cast<int64_t>(0)) : 0;
    // inclusive sums of all three over the warp, exclusive ones of the warps' totals by warp 0
    int64_t n = need, c = count;
    int32_t f = __popc(free_bits);
    auto warp_sums = [&](int64_t &x, int64_t &y, int32_t &z) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t ux = __shfl_up_sync(0xffffffffu, x, o), uy = __shfl_up_sync(0xffffffffu, y, o);
            const int32_t uz = __shfl_up_sync(0xffffffffu, z, o);
            if (lane >= o) {
                x += ux;
                y += uy;
                z += uz;
            }
        }
    };
    warp_sums(n, c, f);
    if (lane == 31) {
        w_need[warp] = n;
        w_count[warp] = c;
        w_free[warp] = f;
    }
    __syncthreads();
    if (warp == 0) {
        int64_t x = w_need[lane], y = w_count[lane];
        int32_t z = w_free[lane];
        const int64_t x0 = x, y0 = y;
        const int32_t z0 = z;
        warp_sums(x, y, z);
        w_need[lane] = x - x0;
        w_count[lane] = y - y0;
        w_free[lane] = z - z0;
        if (lane == 31) {
            w_count[kOneWarps] = y;
            w_free[kOneWarps] = z;
        }
    }
    __syncthreads();
    n += w_need[warp];
    c += w_count[warp];
    int32_t rank = w_free[warp] + f - __popc(free_bits);
    const int64_t out0 = c - count, tokens = w_count[kOneWarps];
    const int32_t free_total = w_free[kOneWarps];
    if (b == 0) s_prefix[0] = cu_new[0] = 0;
    if (b < B) {
        s_prefix[b + 1] = static_cast<int32_t>(min(n, static_cast<int64_t>(INT32_MAX)));
        cu_new[b + 1] = static_cast<int32_t>(min(c, static_cast<int64_t>(INT32_MAX)));
        s_cu[b] = static_cast<int32_t>(min(out0, static_cast<int64_t>(INT32_MAX)));
        s_start[b] = static_cast<int32_t>(g.start);
        s_end[b] = static_cast<int32_t>(g.end);
    }
    __syncthreads();
    // The sequence's own part: slots in the block held already, or -1 where it gets nothing
    if (b < B) {
        int bits = (g.valid ? 0 : PKV_ERRBIT_CONTEXT) | (c > num_slots_out ? PKV_ERRBIT_SPAN : 0);
        int32_t *row = block_tables + static_cast<int64_t>(b) * max_blocks;
        int64_t upto = g.end;  // slots of [start, upto)
        int32_t id = -1;
        if (g.valid && (need == 0 || n <= free_total)) {
            upto = min(g.end, g.held * bs);
            if (upto > g.start) {
                id = row[g.held - 1];
                if (id < 0 || id >= num_blocks) {
                    id = -1;
                    bits |= PKV_ERRBIT_BLOCK_RANGE;
                }
            }
        } else if (g.valid) {
            for (int64_t j = g.held; j < g.grown; ++j) row[j] = -1;
            bits |= PKV_ERRBIT_NO_BLOCKS;
        }
        const int64_t stop = min(upto, g.start + max(num_slots_out - out0, static_cast<int64_t>(0)));
        // the start's slot, where id is a block
        uint32_t at = static_cast<uint32_t>(id * static_cast<int64_t>(bs) + g.start - (g.held - 1) * bs);
        for (int64_t p = g.start; p < stop; ++p, ++at) slots[out0 + p - g.start] = id < 0 ? -1 : static_cast<int32_t>(at);
        if (bits && err_flag) atomicOr(err_flag, bits);
    }
    for (int64_t k = tokens + b; k < num_slots_out; k += kOneThreads) slots[k] = -1;  // padding
    // The granted blocks, the largest prefix of the needs that the free blocks cover
    const int32_t granted = s_prefix[last_at_most(s_prefix, B, free_total)];
    for (int32_t r0 = 0; r0 < granted; r0 += kOneThreads) {
        for (; free_bits && rank < min(r0 + kOneThreads, granted); ++rank, free_bits &= free_bits - 1)
            e_id[rank - r0] = 32 * b + __ffs(free_bits) - 1;
        __syncthreads();
        const int32_t taken = min(kOneThreads, granted - r0), span = min(bs, num_slots_out);
        if (b < taken) {
            const int32_t r = r0 + b, id = e_id[b], to = last_at_most(s_prefix, B, r);
            const Growth h = growth_of(s_start[to], s_end[to], bs, max_blocks);
            const int64_t j = h.held + r - s_prefix[to];
            ref_counts[id] = 1;
            block_tables[static_cast<int64_t>(to) * max_blocks + j] = id;
            const int64_t at = s_cu[to] + j * bs - h.start;
            e_out[b] = static_cast<int32_t>(min(at, static_cast<int64_t>(num_slots_out)));
            e_len[b] = static_cast<int32_t>(min(static_cast<int64_t>(bs), h.end - j * bs));
        }
        __syncthreads();
        for (int32_t x = b; x < taken * span; x += kOneThreads) {  // span: what the slot map can hold, at most kOneTokens
            const int32_t e = x / span, o = x - e * span;
            if (o < e_len[e] && o < num_slots_out - e_out[e]) slots[e_out[e] + o] = e_id[e] * bs + o;
        }
        __syncthreads();  // the entries are read before the next ones overwrite them
    }
}

// One CTA per sequence: table entries of the blocks that hold positions
// [keep, len) only go back; a block is free again when its count reaches 0.
// Each entry is a load and an atomic that waits for it, so the entries of a long
// sequence are spread over the threads.
__global__ void __launch_bounds__(kShrinkThreads)
table_shrink_kernel(int32_t *__restrict__ block_tables, int32_t max_blocks, const int32_t *__restrict__ keeps,
                    const int32_t *__restrict__ lens, int32_t bs, int32_t *__restrict__ ref_counts,
                    int32_t num_blocks, int32_t *__restrict__ err_flag) {
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.x;
    const Growth g = growth_of(keeps[b], lens[b], bs, max_blocks);
    if (!g.valid) {
        if (threadIdx.x == 0 && err_flag) atomicOr(err_flag, PKV_ERRBIT_CONTEXT);
        return;
    }
    int32_t *row = block_tables + static_cast<int64_t>(b) * max_blocks;
    int bits = 0;
    for (int64_t j = g.held + threadIdx.x; j < g.grown; j += kShrinkThreads) {
        const int32_t id = row[j];
        if (id == -1) continue;  // never granted, or given back already
        row[j] = -1;
        if (id < 0 || id >= num_blocks) {
            bits |= PKV_ERRBIT_BLOCK_RANGE;
        } else if (atomicSub(ref_counts + id, 1) <= 0) {  // not referenced: the count stays as it was
            atomicAdd(ref_counts + id, 1);
            bits |= PKV_ERRBIT_REF_COUNT;
        }
    }
    if (bits && err_flag) atomicOr(err_flag, bits);
}

int32_t table_chunk(int32_t num_blocks) {
    const int64_t per = (static_cast<int64_t>(num_blocks) + kMaxTabChunks - 1) / kMaxTabChunks;
    return static_cast<int32_t>(per <= kTabThreads ? kTabThreads : (per + kTabThreads - 1) / kTabThreads * kTabThreads);
}

pkv_status check_table_sizes(const char *who, int32_t max_blocks, int32_t num_seqs, int32_t block_size,
                             int32_t num_blocks) {
    if (max_blocks < 0 || num_seqs < 0 || block_size <= 0 || num_blocks < 0)
        return set_error(PKV_ERR_INVALID_ARG, "%s: bad sizes", who);
    if (static_cast<int64_t>(num_blocks) * block_size > INT32_MAX)
        return set_error(PKV_ERR_INVALID_ARG, "%s: num_blocks * block_size >= 2^31", who);
    if (num_seqs > 65535) return set_error(PKV_ERR_UNSUPPORTED, "%s: more than 65535 sequences in one call", who);
    return PKV_OK;
}

bool grows_alone(int32_t num_seqs, int32_t num_blocks, int64_t num_new_tokens) {
    return num_seqs <= kOneSeqs && num_blocks <= kOneBlocks && num_new_tokens <= kOneTokens;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_grow_block_tables_workspace_size(int32_t num_seqs, int32_t num_blocks, int64_t num_new_tokens) {
    if (num_seqs <= 0 || num_blocks < 0 || grows_alone(num_seqs, num_blocks, num_new_tokens)) return 0;
    return round256((static_cast<size_t>(num_seqs) + 1) * 4) + round256(kMaxTabChunks * 4);
}

extern "C" pkv_status pkv_grow_block_tables(int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *starts,
                                            const int32_t *ends, int32_t num_seqs, int32_t block_size,
                                            int32_t *ref_counts, int32_t num_blocks, int32_t *cu_new,
                                            int32_t *slot_mapping, int64_t num_new_tokens, void *workspace,
                                            size_t workspace_bytes, int32_t *err_flag, void *stream) {
    const pkv_status chk = check_table_sizes("grow", max_blocks_per_seq, num_seqs, block_size, num_blocks);
    if (chk != PKV_OK) return chk;
    if (num_new_tokens < 0) return set_error(PKV_ERR_INVALID_ARG, "grow: num_new_tokens < 0");
    if (num_seqs == 0) return ok();
    if (!starts || !ends || !cu_new || (max_blocks_per_seq > 0 && !block_tables) || (num_blocks > 0 && !ref_counts) ||
        (num_new_tokens > 0 && !slot_mapping))
        return set_error(PKV_ERR_INVALID_ARG, "grow: NULL pointer");
    if (grows_alone(num_seqs, num_blocks, num_new_tokens)) {
        const cudaError_t e = launch_pdl(kPdlSlotMapping, table_grow_one_kernel, dim3(1), dim3(kOneThreads), 0,
                                         static_cast<cudaStream_t>(stream), block_tables, max_blocks_per_seq, starts, ends,
                                         num_seqs, block_size, ref_counts, num_blocks, cu_new, slot_mapping,
                                         static_cast<int32_t>(num_new_tokens), err_flag);
        if (e != cudaSuccess) return set_error(PKV_ERR_CUDA, "grow launch: %s", cudaGetErrorString(e));
        return ok();
    }
    const size_t need = pkv_grow_block_tables_workspace_size(num_seqs, num_blocks, num_new_tokens);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 256))
        return set_error(PKV_ERR_WORKSPACE, "grow: workspace needs %zu bytes (256-byte aligned), got %zu", need,
                         workspace_bytes);
    auto prefix = static_cast<int32_t *>(workspace);
    auto chunk_free = reinterpret_cast<int32_t *>(static_cast<char *>(workspace) +
                                                  round256((static_cast<size_t>(num_seqs) + 1) * 4));
    const int32_t chunk = table_chunk(num_blocks);
    const int32_t chunks = static_cast<int32_t>((static_cast<int64_t>(num_blocks) + chunk - 1) / chunk);
    auto s = static_cast<cudaStream_t>(stream);
    cudaError_t e = launch_pdl(kPdlSlotMapping, table_count_kernel, dim3(1 + chunks), dim3(kTabThreads), 0, s, starts,
                               ends, num_seqs, block_size, max_blocks_per_seq, ref_counts, num_blocks, chunk, prefix,
                               chunk_free, cu_new, err_flag);
    if (e == cudaSuccess)
        e = launch_pdl(kPdlSlotMapping, table_assign_kernel, dim3(chunks + (num_seqs + kTabWarps - 1) / kTabWarps),
                       dim3(kTabThreads), 0, s, block_tables, max_blocks_per_seq, starts, ends, num_seqs, block_size,
                       ref_counts, num_blocks, chunk, chunks, prefix, chunk_free, cu_new, slot_mapping,
                       num_new_tokens, err_flag);
    if (e != cudaSuccess) return set_error(PKV_ERR_CUDA, "grow launch: %s", cudaGetErrorString(e));
    return ok();
}

extern "C" pkv_status pkv_shrink_block_tables(int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *keeps,
                                              const int32_t *lens, int32_t num_seqs, int32_t block_size,
                                              int32_t *ref_counts, int32_t num_blocks, int32_t *err_flag,
                                              void *stream) {
    const pkv_status chk = check_table_sizes("shrink", max_blocks_per_seq, num_seqs, block_size, num_blocks);
    if (chk != PKV_OK) return chk;
    if (num_seqs == 0) return ok();
    if (!keeps || !lens || (max_blocks_per_seq > 0 && !block_tables) || (num_blocks > 0 && !ref_counts))
        return set_error(PKV_ERR_INVALID_ARG, "shrink: NULL pointer");
    const cudaError_t e = launch_pdl(kPdlSlotMapping, table_shrink_kernel,
                                     dim3(num_seqs), dim3(kShrinkThreads), 0, static_cast<cudaStream_t>(stream),
                                     block_tables, max_blocks_per_seq, keeps, lens, block_size, ref_counts,
                                     num_blocks, err_flag);
    if (e != cudaSuccess) return set_error(PKV_ERR_CUDA, "shrink launch: %s", cudaGetErrorString(e));
    return ok();
}
