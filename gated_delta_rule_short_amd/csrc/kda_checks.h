// kda_checks.h -- argument checks shared by the entry points (host code).
//
// A check that fails leaves its message in the calling thread's buffer
// (kda_last_error) and returns the status.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kda.h"

namespace kda {
namespace checks {

// Stores the calling thread's message and returns st; clear_error empties it.
kda_status fail(kda_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
void clear_error();

inline kda_status hip_fail(hipError_t e, const char *what) {
    return fail(KDA_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

inline size_t esize(kda_dtype d) { return d == KDA_BF16 ? 2 : 4; }
inline size_t state_esize(uint32_t flags) { return (flags & KDA_F_STATE_BF16) ? 2 : 4; }

inline bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const char *pa = static_cast<const char *>(a), *pb = static_cast<const char *>(b);
    return pa < pb + nb && pb < pa + na;
}

// Checks an optional host copy of cu_seqlens.
inline kda_status check_cu_host(const int32_t *cu, int32_t n, int64_t total) {
    if (!cu) return KDA_OK;
    if (cu[0] != 0) return fail(KDA_ERR_INVALID_ARG, "cu_seqlens[0] = %d, expected 0", cu[0]);
    for (int32_t i = 0; i < n; ++i)
        if (cu[i + 1] < cu[i])
            return fail(KDA_ERR_INVALID_ARG, "cu_seqlens not monotone at %d (%d > %d)", i, cu[i],
                        cu[i + 1]);
    if ((int64_t)cu[n] != total)
        return fail(KDA_ERR_INVALID_ARG, "cu_seqlens[%d] = %d, expected total_tokens = %lld", n,
                    cu[n], (long long)total);
    return KDA_OK;
}

// Rows of the state and conv-state arrays: the pool size with a slot map, else
// one per sequence.
inline kda_status pool_rows(const int32_t *slots, int32_t num_slots, int32_t num_seqs, size_t &rows) {
    if (!slots) {
        rows = (size_t)num_seqs;
        return KDA_OK;
    }
    if (num_slots < 1) return fail(KDA_ERR_INVALID_ARG, "state_slots needs num_slots >= 1");
    rows = (size_t)num_slots;
    return KDA_OK;
}

// A call's buffers as (pointer, bytes, name); the first `n_written` are written
// by the call.  Every written buffer must overlap no other buffer of the call.
// NULL or empty buffers overlap nothing; an allowed in-place pair is passed with
// the input side's size set to 0.
struct Buf {
    const void *p;
    size_t bytes;
    const char *name;
};
inline kda_status check_written(const Buf *b, int n, int n_written) {
    for (int i = 0; i < n_written; ++i)
        for (int j = 0; j < n; ++j) {
            if (j == i || (j < n_written && j < i)) continue;
            if (overlap(b[i].p, b[i].bytes, b[j].p, b[j].bytes))
                return fail(KDA_ERR_INVALID_ARG, "%s overlaps %s", b[i].name, b[j].name);
        }
    return KDA_OK;
}

}  // namespace checks
}  // namespace kda
