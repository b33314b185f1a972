// Argument checks that the operators' C entry points share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "gdn.h"

namespace gdn {
namespace checks {

constexpr size_t kAlign = 256;
constexpr int kMaxT = 1 << 30;

inline size_t round_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
inline bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
inline bool off_elem(const void* p, int dtype) { return reinterpret_cast<uintptr_t>(p) % (dtype == GDN_F32 ? 4 : 2) != 0; }

inline gdn_status check_dense(std::initializer_list<const void*> ptrs) {
    for (const void* p : ptrs)
        if (p && off16(p)) return GDN_ERR_MISALIGNED;
    return GDN_OK;
}
inline gdn_status check_cu(const int32_t* cu) { return reinterpret_cast<uintptr_t>(cu) & 3u ? GDN_ERR_MISALIGNED : GDN_OK; }

// A strided input: present, aligned to its element, rows at least `row` apart.
inline gdn_status check_rows(const void* p, int64_t stride, int64_t row, int dtype) {
    if (!p || stride < row || stride >= (1LL << 40)) return GDN_ERR_INVALID_ARG;
    return off_elem(p, dtype) ? GDN_ERR_MISALIGNED : GDN_OK;
}

inline gdn_status check_ws(const void* p, size_t bytes, size_t need) {
    if (need == 0) return GDN_OK;
    if (!p || bytes < need) return GDN_ERR_INVALID_ARG;
    return reinterpret_cast<uintptr_t>(p) & (kAlign - 1) ? GDN_ERR_MISALIGNED : GDN_OK;
}

// Tokens of a call: B rows of T, or (packed: B sequences) T in all.
inline long long token_count(int B, int T, bool varlen) { return varlen ? T : static_cast<long long>(B) * T; }

inline gdn_status check_sizes(int B, int T, int D, int dtype, bool varlen) {
    if (B < 1 || T < 0 || D < 1) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_F32) return GDN_ERR_INVALID_ARG;
    if (B > 65535 || T > kMaxT || D > 65536) return GDN_ERR_UNSUPPORTED;
    if (token_count(B, T, varlen) >= (1LL << 40) / D) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

#define GDN_TRY(expr)                          \
    do {                                       \
        const gdn_status st_ = (expr);         \
        if (st_ != GDN_OK) return st_;         \
    } while (0)

}  // namespace checks
}  // namespace gdn
