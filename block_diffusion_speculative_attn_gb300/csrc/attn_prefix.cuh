// attn_prefix.cuh -- what the two kernels of a shared-prefix call agree on: which
// keys of a request belong to its group's prefix, the prefix work units with
// their cost offsets, and where the partials of a unit's pieces are.
//
// Group g holds requests [off[g], off[g + 1]) and shares its first
// P' = floor(P_g / 128) * 128 keys.  Its query rows of one KV head, (token, head
// of the group) in token order, are cut into tiles of npt whole tokens (at most
// kPrefixRows rows), two tiles to a pair.  CTAs work in teams of T (1 or 2): a team
// takes T pairs of one KV head over the same keys, a pair a member.  A unit is a
// team's T pairs over all P' keys, numbered (group, KV head, T pairs); each is
// charged kPrefixUnitCost virtual tiles and its P' / 128 real ones, and team b of S
// takes the cost range [b Wc / S, (b + 1) Wc / S).  The piece that holds a unit's
// first tile goes to per-row buffers (a row has one such piece), with the numbers of
// the teams that hold the unit's first and last tile; any other piece is the first of
// its CTA and goes to that CTA's slot.
#pragma once

#include "attn_common.cuh"
#include "bdsa_internal.h"

namespace bdsa {
namespace {

constexpr int kPrefixRows = 128;     // query rows of a tile
// Virtual tiles a unit switch is charged (a Q load, an epilogue; with one, three and
// four the cases below are within 3%).
constexpr int kPrefixUnitCost = 2;
// A team takes at least this cost: below it the pieces' partials and their merge
// cost more than the CTAs gain (64 single tokens of 32 heads behind 2048 keys 63 us a
// call; with 3 and 4 tiles 66, 8: 67, 12: 69; longer prefixes do not care).
constexpr int kPrefixMinCost = 6;

// The keys of request r (length L) its group shares, in whole tiles; g its
// group, or -1 (and 0 keys) when the groups do not place it or its prefix is
// not inside its length.
__device__ __forceinline__ int request_prefix(const PrefixParams &x, int r, int L, int &g) {
    int lo = 0, hi = x.ng;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(x.group_offsets + mid) <= r) lo = mid;
        else hi = mid;
    }
    const int P = __ldg(x.prefix_lens + lo);
    const bool ok = __ldg(x.group_offsets + lo) <= r && r < __ldg(x.group_offsets + lo + 1) &&
                    __ldg(x.group_offsets + lo) >= 0 && P >= 0 && P <= L;
    g = ok ? lo : -1;
    return ok ? P & ~(kBN - 1) : 0;
}

// Group g's first request, tokens and shared tiles (no tokens when its bounds
// are not within [0, bs], or no row can hold its prefix).
__device__ __forceinline__ void group_shape(const PrefixParams &x, int g, int B, int &r0,
                                            int &tokens, int &nt) {
    const int o0 = __ldg(x.group_offsets + g), o1 = __ldg(x.group_offsets + g + 1);
    const int P = __ldg(x.prefix_lens + g);
    const bool ok = o0 >= 0 && o0 < o1 && o1 <= x.bs && P >= kBN && P <= x.max_keys;
    r0 = ok ? o0 : 0;
    tokens = ok ? (o1 - o0) * B : 0;
    nt = ok ? P / kBN : 0;
}
__device__ __forceinline__ int group_pairs(const PrefixParams &x, int tokens) {
    return (tokens + 2 * x.npt - 1) / (2 * x.npt);
}

// Units of a group and KV head, by teams of T.
__device__ __forceinline__ int group_units(const PrefixParams &x, int tokens, int T) {
    return (group_pairs(x, tokens) + T - 1) / T;
}

__device__ __forceinline__ long long prefix_range_start(long long b, long long Wc, long long S) {
    return b * Wc / S;
}

// A block row's place in its group (nt 0: nothing shared).
struct PrefixRow {
    int nt;    // shared tiles
    int pair;  // the row's pair
    int row;   // the block row's first row within the pair's 2 * kPrefixRows
};
__device__ __forceinline__ PrefixRow prefix_row(const PrefixParams &x, int g, int r, int i_blk,
                                                int B, int G) {
    PrefixRow u{0, 0, 0};
    if (g < 0) return u;
    int r0, tokens;
    group_shape(x, g, B, r0, tokens, u.nt);
    const int t = (r - r0) * B + i_blk;  // token within the group
    const int tile = t / x.npt;
    u.pair = tile >> 1;
    u.row = (tile & 1) * kPrefixRows + (t - tile * x.npt) * G;
    return u;
}

// The team whose cost range holds cost c: the largest b with b Wc / S <= c (an fp32
// estimate, then exact steps: 64-bit division is a long subroutine here).
__device__ __forceinline__ int prefix_team_of(long long c, long long Wc, int S) {
    int b = (int)((float)(c + 1) * (float)S / (float)Wc);
    b = max(0, min(b, S - 1));
    while (b > 0 && b * Wc > c * S + S - 1) --b;
    while (b + 1 < S && (b + 1) * Wc <= c * S + S - 1) ++b;
    return b;
}

}  // namespace
}  // namespace bdsa
