// The 4-bit cache: where a token's keys and values lie, and who they belong to.
//
// Sixteen consecutive tokens of one kv head form a group of 18 W bytes (W = 64, 128
// or 256 elements a head): [K codes 8 W | V codes 8 W | K scales W | V scales W].
// A page holds page / 16 groups of each head, [head][group], so that a page's tokens
// of a head are one run of bytes that a bulk copy moves.
//
// Inside a group the order is that of the attention's 16-bit matrix fragments
// (m16n8k16; lane = 4 g + c), so that each lane reads what it multiplies with wide,
// conflict-free loads:
//   K: token t = 8 half + g, elements in chunks of 16 bytes (8 where W is 64), chunk c
//      of 128 (64) elements: the lane's elements of one token are its k indices.
//      Scales: the lane's of both halves side by side.
//   V: tokens 8 half + 2 c + e (e = 0, 1) are a k pair of the lane, elements g W/8 .. are its
//      n indices: a byte per element, token e = 0 in its low four bits, in lines of 16 bytes
//      (8 where W is 64) a lane.  Scales: [block][c][half][e].
#pragma once
#include <cstdint>

#include "h3fp4_token.h"

namespace h3fp4 {

template <int W>
struct CacheLayout {
    static constexpr int kGroupBytes = 18 * W;
    static constexpr int kV = 8 * W, kKScale = 16 * W, kVScale = 17 * W;
    static constexpr int kBlocks = W / 16;

    // The eight code bytes of elements [16 b, 16 b + 16) of token t: K.
    static __device__ __forceinline__ int k_codes(int t, int b)
    {
        return W == 64 ? t * 32 + b * 8 : (b >> 3) * 1024 + t * 64 + (b & 7) * 8;
    }
    static __device__ __forceinline__ int k_scale(int t, int b)
    {
        const int g = t & 7, half = t >> 3;
        if (W == 64) return kKScale + (g * 4 + b) * 2 + half;
        if (W == 128) return kKScale + ((g * 4 + (b >> 1)) * 2 + half) * 2 + (b & 1);
        return kKScale + ((g * 4 + ((b & 7) >> 1)) * 2 + half) * 4 + (b >> 3) * 2 + (b & 1);
    }
    // V: 16 bytes of elements [16 b, 16 b + 16), shared by two tokens (W = 64: eight at each of two
    // places, the second at + 32); token t's are their low or, for odd t, high four bits.
    static __device__ __forceinline__ int v_codes(int t, int b)
    {
        const int half = t >> 3, c = (t & 7) >> 1;
        if (W == 64) return kV + half * 256 + (8 * b + c) * 8;
        if (W == 128) return kV + half * 512 + (4 * b + c) * 16;
        return kV + half * 1024 + (b & 1) * 512 + (4 * (b >> 1) + c) * 16;
    }
    static __device__ __forceinline__ int v_scale(int t, int b)
    {
        return kVScale + (b * 4 + ((t & 7) >> 1)) * 4 + (t >> 3) * 2 + (t & 1);
    }
};

// The sequence of packed row r, or -1 where it is none's: one warp, all lanes.
__device__ __forceinline__ int cache_sequence(const CacheView& c, long long r, int lane)
{
    if (!c.row_off) return (int)r;
    if (r < c.row_off[0]) return -1;
    int s = 0;
    for (int i = 0; i < c.nseq; i += 32) {
        const bool behind = i + lane < c.nseq && c.row_off[i + lane + 1] <= r;
        s += __popc(__ballot_sync(0xffffffffu, behind));
    }
    return s < c.nseq ? s : -1;
}

// Tokens of sequence s that the table has room for.
__device__ __forceinline__ long long cache_length(const CacheView& c, int s)
{
    const long long room = c.max_pages * c.page, n = c.length[s];
    return n < 0 ? 0 : n < room ? n : room;
}

// The group of 16 tokens that holds position pos of sequence s and head h, or null where
// the table names no page of the pool.
template <int W>
__device__ __forceinline__ uint8_t* cache_group(const CacheView& c, int s, long long pos, int h)
{
    const long long page = c.table[(long long)s * c.max_pages + pos / c.page];
    if (page < 0 || page >= c.n_pages) return nullptr;
    const int groups = c.page / kCacheGroup;
    return c.pool + ((page * c.Hkv + h) * groups + (pos % c.page) / kCacheGroup) * CacheLayout<W>::kGroupBytes;
}

}  // namespace h3fp4
