// What the shared prefix's kernel and paged attention's kernel behind it have
// to agree on: groups of sequences, and which part of the GPU each takes.
//
// Where the prefix has blocks of two row tiles, the tensor cores are what it waits for, and the two run side
// by side: the first has one CTA per SM, those of them that have work keep their SM, and the second's
// CTAs start on the SMs that the others left (64 sequences of 32 heads behind 4,096 cells, 580
// cells of their own each: 55 us one after the other, 48 so; 512 of 16 heads behind 8,192, 72 of their own: 66 and 60).
// Blocks of one row tile want all of the bandwidth, and so do the own cells: side by side they were slower (32
// sequences behind 65,536 cells 63 us, 68 so). Lengths are on the device, so each kernel finds the division itself.
#pragma once

#include "cache_internal.cuh"
#include "ptx.cuh"

namespace qsa {

constexpr int PREFIX_TILE = 128;   // prefix cells of a tile

// A group of sequences.
struct PrefixGroup {
    int first, count, len, tiles, blocks;   // blocks of rows
};
__device__ __forceinline__ PrefixGroup prefix_group(const PrefixShare &p, int g) {
    PrefixGroup x;
    x.first = min(max(ld_in(p.cu + g), 0), p.nseq);
    x.count = min(max(ld_in(p.cu + g + 1), x.first), p.nseq) - x.first;
    x.len = min(max(ld_in(p.prefix_lens + g), 0), p.capacity);
    x.tiles = (x.len + PREFIX_TILE - 1) / PREFIX_TILE;
    x.blocks = (x.count + p.block - 1) / p.block;
    return x;
}
// Of all KV heads.
__device__ __forceinline__ long long prefix_tiles(const PrefixShare &p, const PrefixGroup &x) {
    return static_cast<long long>(x.tiles) * x.blocks * p.nkv;
}
// The time (ns) that they take one CTA.
__device__ __forceinline__ long long prefix_work(const PrefixShare &p, const PrefixGroup &x) {
    return prefix_tiles(p, x) * (x.count > p.seqs ? p.two_tiles_ns : p.one_tile_ns);
}

// CTAs (and SMs) for the prefix's `tiles` and `work`, where the sequences' own cells are `own_tiles` tiles
// of paged attention, whose kernel takes two CTAs on each of the other SMs: the fewest whose time is no longer than
// the other kernel's, by what each was measured to take to begin and end, and per tile; all SMs where they do not
// run side by side. Found by a whole warp.
__device__ __forceinline__ int prefix_ctas(const PrefixShare &p, long long tiles, long long work, long long own_tiles) {
    constexpr float START_NS = 4000.0f;    // the prefix's kernel takes so much longer to begin and end
    const int most = static_cast<int>(min(tiles, static_cast<long long>(p.grid)));
    const float w = static_cast<float>(work);
    if (own_tiles == 0 || 2.0f * w < static_cast<float>(tiles) * static_cast<float>(p.one_tile_ns + p.two_tiles_ns)) return p.sms;
    const float own = 0.5f * (static_cast<float>(own_tiles) * p.own_tile_ns + static_cast<float>(p.own_units) * p.own_unit_ns);
    const int lane = threadIdx.x & 31;
    int lo = min(1, most), hi = most;      // the answer, if below `most`, lies in lo .. hi - 1
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32, c = lo + (lane + 1) * step - 1;
        const bool enough = c >= hi || c >= p.sms ||
                            START_NS + __fdividef(w, static_cast<float>(c)) <= __fdividef(own, static_cast<float>(p.sms - c));
        const int first = __ffs(__ballot_sync(FULL_MASK, enough)) - 1;   // the last lane's c is at least hi - 1
        if (first < 0) return hi;
        hi = min(hi, lo + (first + 1) * step - 1);
        lo += first * step;
        if (step == 1) break;
    }
    return hi;
}

}  // namespace qsa
