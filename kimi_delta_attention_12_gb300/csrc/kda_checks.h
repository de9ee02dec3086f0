// kda_checks.h -- the argument checks the C-ABI translation units share.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/kda.h"

namespace kda {

inline bool aligned(const void* p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

inline bool supported_dim(int32_t d) { return d == 32 || d == 64 || d == 128; }

inline size_t elem_bytes(kda_dtype dt) { return dt == KDA_F32 ? 4 : 2; }

inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Whether the byte ranges [a, a + na) and [b, b + nb) share a byte.
inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// A host mirror of cu_seqlens starts at 0, does not decrease and ends at total_T; without
// cu_seqlens itself (`equal`) the sequences are N of equal length, and it says so too.
inline bool valid_host_seqlens(const int32_t* cu, int32_t N, int32_t total_T, bool equal) {
    if (cu[0] != 0 || cu[N] != total_T) return false;
    for (int32_t n = 0; n < N; ++n) {
        if (cu[n + 1] < cu[n] || (equal && cu[n + 1] - cu[n] != total_T / N)) return false;
    }
    return true;
}

}  // namespace kda
