// host.h — what the library's host translation units share: error reporting,
// per-device state, tensor-map encoding and per-(device, stream) workspaces
// (all defined in api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <mutex>

#include "internal.h"
#include "tmg.h"

namespace tmg {

struct DeviceState {
    bool ready = false;
    int num_sms = 0;
    int cc_major = 0, cc_minor = 0;
    uint32_t *err_word = nullptr;
};

// Set the calling thread's last error message and return `st`.
tmg_status fail(tmg_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
tmg_status cuda_fail(cudaError_t e, const char *what);
void clear_error();

// State of the current device (set up on first use).
tmg_status device_state(DeviceState **out);
ErrCtx err_ctx(const DeviceState &ds);

// One line on stderr when TMG_LOG is set.
void log_choice(const char *fmt, ...) __attribute__((format(printf, 1, 2)));

// A tiled tensor map of `rank` dimensions: dims[i] extents (innermost first),
// strides[i] bytes between elements of dimension i + 1, box[i] extents of one
// copy (inner extent of 32, 64 or 128 bytes, swizzled over as many); out-of-range
// elements read as zero and are not written.  reread: many tiles read each
// element.  Encoded anew on every call.
tmg_status encode_nd(CUtensorMap *map, CUtensorMapDataType dt, int rank, const void *base, const int64_t *dims,
                     const int64_t *strides, const int *box, bool reread = false);

// Workspaces per (device, stream), grown on demand; an outgrown one that a captured
// graph may name is kept until tmg_shutdown.
enum Workspace {
    // the grouped products, the dense product with the residual epilogue, routing
    kWsPackA,          // operand copies with 16-byte rows
    kWsPackB,
    kWsGather,         // rows gathered by number
    kWsPartials,       // fp32 partial tiles of split contractions
    kWsCounters,       // arrival counters: zero on entry, zero again on exit
    kWsRoute,          // per-block expert counts of the routing plan
    kWsGrad,           // dz of the dense product's gradient and its column partials
    // the other GEMM paths, which the dense product's gradient takes too
    kWsTc2Partials,    // pair kernel: stream-K partial tiles and tile counters
    kWsTc2Counters,
    kWsSkinnyPartials, // skinny kernel: the same
    kWsSkinnyCounters,
    kWsLayoutA,        // general layouts: packed A, packed B, dense D
    kWsLayoutB,
    kWsLayoutD,
    kWsMxScales,       // MXFP4 scales in chunk order
    kWsCount
};
void *workspace(Workspace which, size_t bytes, cudaStream_t s, tmg_status *st);

// Held by an entry point from its first workspace to its last launch: another host
// thread's call on the same stream must not come between the kernel that fills a
// workspace and the one that reads it.  Recursive: entry points call one another.
class StreamLock {
public:
    explicit StreamLock(cudaStream_t s);
    ~StreamLock() { mu_->unlock(); }
    StreamLock(const StreamLock &) = delete;
    StreamLock &operator=(const StreamLock &) = delete;

private:
    std::recursive_mutex *mu_;
};

}  // namespace tmg
