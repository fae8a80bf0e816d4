// kv_host.h -- host-side helpers that the entry points of kv_api.cu and
// kv_chunk_api.cu share: argument checks, the device status word, the
// tensor-map encoder.  Defined in kv_api.cu.
#pragma once

#include <cudaTypedefs.h>
#include <stddef.h>
#include <stdint.h>

#include "kvsparse.h"

namespace kvs {

int current_device();       // -1 when there is none
int *status_ptr(int dev);   // the device's status word, null when it cannot be found
int sm_count(int dev);
int check_shape(const kv_shape *s);
// device-visible address of a cache array, checked against the shape's kv_loc
int resolve_kv(const kv_shape *s, const void *p, const void **dev_ptr);
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // null when the driver has none
// testing hooks set by kv_debug_config
int debug_skip_page();
unsigned long long wait_limit_ns();

inline bool al16(const void *p) { return p && ((uintptr_t)p & 15u) == 0; }
inline bool al4(const void *p) { return p && ((uintptr_t)p & 3u) == 0; }
inline int elem_bytes(int dtype) { return dtype == KV_F32 ? 4 : 2; }
inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace kvs
