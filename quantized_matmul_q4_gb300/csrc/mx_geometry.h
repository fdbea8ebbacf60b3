// Launch geometry of the MX products: plain host C++ (no CUDA types), so that
// the CPU tests compile this same header and check it.
#pragma once

namespace q4mm {

// CTAs that share a tile's K: as many as fill the SMs with two CTAs each, at
// most 8 (a portable cluster) and two stages of K to each.
inline int mx_split(int row_tiles, int tok_tiles, int stages, int num_sms) {
    const long long tiles = (long long)row_tiles * tok_tiles;
    int S = 1;
    while (S < 8 && tiles * (S + 1) <= 2LL * num_sms && 2 * (S + 1) <= stages) ++S;
    return S;
}

}  // namespace q4mm
