// api_internal.h -- what the entry points in different files share: the
// calling thread's error record, the per-device set-up of api.cu, and the
// library's stream-ordered workspace.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "libmla.h"

namespace mla {

// Records the message as the calling thread's last error (mla_last_error) and returns `status`.
int report_error(int status, const char *msg);
int report_errorf(int status, const char *fmt, ...);
int report_cuda(cudaError_t e, const char *what);

// The current device's set-up (architecture check included): its error word and SM count.
struct DeviceInfo {
    int *err_word;
    int sm_count;
};
int device_info(DeviceInfo *out);

// The library's workspace of (current device, stream), at least `need` bytes; see mla_decode_fwd.
int stream_workspace(size_t need, cudaStream_t stream, void **ws, size_t *ws_bytes);

// Tensor map over a 16-bit (elem 2) or 8-bit (elem 1) tensor of four dimensions, innermost
// first; strides in bytes of dimensions 1 to 3.
int encode_map_4d(CUtensorMap *map, int elem, const void *base, const uint64_t dims[4], const uint64_t strides[3],
                  const uint32_t box[4], CUtensorMapSwizzle swizzle);

// Whether rows of `extent` elements, n[i] of them at stride s[i] in each of `dims` dimensions, share no element: by rising
// stride, each dimension of more than one entry must step past all that the ones before it span.  (Layouts that
// interleave their dimensions without such an order are taken to overlap.)
inline bool rows_apart(const int64_t *n, const int64_t *s, int dims, int64_t extent) {
    __int128 span = extent;
    for (int left = (1 << dims) - 1; left;) {
        int k = -1;   // the dimension of the smallest stride that is left
        for (int i = 0; i < dims; ++i)
            if ((left >> i & 1) && (k < 0 || s[i] < s[k])) k = i;
        left &= ~(1 << k);
        if (n[k] <= 1) continue;
        if (s[k] < span) return false;
        span += (__int128)(n[k] - 1) * s[k];
    }
    return true;
}

inline bool is_aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace mla
