// experts.h -- rows that lie expert by expert (internal).
//
// Expert e's rows are offsets[e] .. offsets[e+1]-1, the offsets in device
// memory, so no launch can know how many tiles of rows there are.  A grid has
// as many blocks as the worst case needs and each block finds its own tile, or
// that there is none for it.  Offsets are not trusted: each is held to `rows`
// and to at least the largest before it, so that no row is out of range and no
// row belongs to two experts whatever they hold.
#ifndef TLC_EXPERTS_H
#define TLC_EXPERTS_H

#include <hip/hip_runtime.h>

#include <stdint.h>

#include <algorithm>

namespace tlc_experts {

constexpr uint64_t kMaxExperts = 65536;

struct Experts {
    const uint64_t* offsets;  // nullptr: one expert has every row
    uint32_t count;
    uint32_t rows;
};

struct Span {
    uint32_t expert, begin, end;  // rows of the expert
};

// Running maximum and running sum over the wavefront's lanes.
__device__ __forceinline__ uint32_t scan_max(uint32_t v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t o = __shfl_up(v, d);
        if (lane >= d) v = max(v, o);
    }
    return v;
}
__device__ __forceinline__ uint32_t scan_add(uint32_t v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}

__device__ __forceinline__ uint32_t held(const Experts& x, uint32_t i) {
    return (uint32_t)min(x.offsets[i], (uint64_t)x.rows);
}

// Rows of expert first + lane; `before` is the largest offset before them and
// becomes the largest up to the 64th's end.
__device__ __forceinline__ void spans(const Experts& x, uint32_t first, uint32_t* before, uint32_t* begin,
                                      uint32_t* end) {
    const uint32_t e = first + (threadIdx.x & 63);
    const uint32_t b = held(x, min(e, x.count)), n = held(x, min(e + 1, x.count));
    *begin = max(scan_max(b), *before);
    *end = max(*begin, n);
    *before = __shfl(*end, 63);
}

// How many tiles of `tile` rows the experts have, each with its own last one.
__device__ __forceinline__ uint32_t tiles_of(const Experts& x, uint32_t tile) {
    if (!x.offsets) return (x.rows + tile - 1) / tile;
    uint32_t sum = 0, before = 0;
    for (uint32_t first = 0; first < x.count; first += 64) {
        uint32_t b, e;
        spans(x, first, &before, &b, &e);
        sum += __shfl(scan_add((e - b + tile - 1) / tile), 63);
    }
    return __builtin_amdgcn_readfirstlane((int)sum);
}

// The expert of tile `want` (below tiles_of) and the tile's rows begin .. end-1,
// end at most `tile` further and inside the expert.
__device__ __forceinline__ Span tile_rows(const Experts& x, uint32_t tile, uint32_t want) {
    if (!x.offsets) return {0, want * tile, min(x.rows, want * tile + tile)};
    Span s = {0, 0, 0};
    uint32_t sum = 0, before = 0;
    for (uint32_t first = 0; first < x.count; first += 64) {
        uint32_t b, e;
        spans(x, first, &before, &b, &e);
        const uint32_t here = (e - b + tile - 1) / tile, upto = sum + scan_add(here);
        const uint64_t found = __ballot(want < upto);
        if (found) {
            const int at = __builtin_ctzll(found);
            const uint32_t skip = (want - (uint32_t)__shfl((int)(upto - here), at)) * tile;
            const uint32_t begin = (uint32_t)__shfl((int)b, at) + skip, end = (uint32_t)__shfl((int)e, at);
            s = {first + at, begin, min(end, begin + tile)};
            break;
        }
        sum = __shfl((int)upto, 63);
    }
    s.expert = __builtin_amdgcn_readfirstlane((int)s.expert);
    s.begin = __builtin_amdgcn_readfirstlane((int)s.begin);
    s.end = __builtin_amdgcn_readfirstlane((int)s.end);
    return s;
}

// All of an expert's rows.
__device__ __forceinline__ Span rows_of(const Experts& x, uint32_t expert) {
    if (!x.offsets) return {0, 0, x.rows};
    uint32_t most = 0;  // the largest offset up to the expert's own
    for (uint32_t i = threadIdx.x & 63; i <= expert; i += 64) most = max(most, held(x, i));
    const uint32_t begin = __shfl(scan_max(most), 63);
    Span s = {expert, begin, max(begin, held(x, expert + 1))};
    s.begin = __builtin_amdgcn_readfirstlane((int)s.begin);
    s.end = __builtin_amdgcn_readfirstlane((int)s.end);
    return s;
}

// All rows of the expert whose turn it is: the longest first, of equally long
// ones the first, so that no long expert is begun when the others end. More than
// 64 experts, whose lengths one wavefront does not hold at once, come in order.
__device__ __forceinline__ Span rows_by_length(const Experts& x, uint32_t turn) {
    if (!x.offsets || x.count > 64) return rows_of(x, turn);
    uint32_t b, e, before = 0, rank = 0;
    spans(x, 0, &before, &b, &e);
    // different for every lane, least for those past the last expert
    const uint32_t key = min(e - b, (1u << 26) - 1) << 6 | (63 - (threadIdx.x & 63));
    for (uint32_t i = 0; i < x.count; i += 8)
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) rank += (uint32_t)__builtin_amdgcn_readlane((int)key, (int)(i + j)) > key;
    const int at = __builtin_ctzll(__ballot(rank == turn));  // a rank is one lane's
    return {(uint32_t)at, (uint32_t)__builtin_amdgcn_readlane((int)b, at),
            (uint32_t)__builtin_amdgcn_readlane((int)e, at)};
}

// Block b's place among `total`: blocks go round the 8 XCDs, and of each 256
// blocks, which run at about the same time, an XCD takes neighbours.
__device__ __forceinline__ uint32_t xcd_place(uint32_t b, uint32_t total) {
    const uint32_t run = b / 256 * 256, i = b - run, per = min(256u, total - run) / 8;
    return run + (i < per * 8 ? i % 8 * per + i / 8 : i);
}

// Block b's place among experts of `tiles` tiles each, whose times differ: every
// XCD takes an eighth of each expert's tiles, neighbours, where they divide so.
__device__ __forceinline__ uint32_t xcd_share(uint32_t b, uint32_t tiles) {
    if (tiles % 8) return b;
    const uint32_t per = tiles / 8, turn = b / 8;
    return turn / per * tiles + b % 8 * per + turn % per;
}

// The most tiles that `rows` rows of `experts` experts can need.
inline uint64_t most_tiles(uint64_t rows, uint64_t experts, uint64_t tile, bool grouped) {
    return grouped ? rows / tile + std::min(rows, experts) : (rows + tile - 1) / tile;
}

}  // namespace tlc_experts

#endif  // TLC_EXPERTS_H
