// pkv_capture_id, pkv_capture_watch and pkv_capture_gone: which graph a stream
// is being captured into, and when that graph is no more, so that a caller can
// keep scratch memory for as long as a graph may use it.
//
// The graph carries a user object whose destructor the runtime calls once the
// graph, its clones and everything instantiated from them are destroyed.  The
// destructor may run on a thread of CUDA's own, where no CUDA call is allowed:
// it only notes the id.
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>
#include <new>
#include <vector>

#include "paged_kv.h"
#include "pkv_internal.h"

namespace {

struct Gone {
  std::mutex mu;
  std::vector<uint64_t> ids;  // room for every watched graph's id is made when it is watched
  size_t watched = 0;
};

// Never destroyed: graphs may outlive the library's static objects.
Gone& gone() {
  static Gone* g = new Gone;
  return *g;
}

struct Watch {
  uint64_t id;
};

void CUDART_CB note(void* p) {
  Watch* w = static_cast<Watch*>(p);
  {
    std::lock_guard<std::mutex> lk(gone().mu);
    gone().ids.push_back(w->id);
  }
  delete w;
}

pkv_status capture_info(void* stream, unsigned long long* id, cudaGraph_t* graph) {
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  *id = 0;
  const cudaError_t e = cudaStreamGetCaptureInfo(static_cast<cudaStream_t>(stream), &status, id, graph, nullptr,
                                                 nullptr, nullptr);
  if (e != cudaSuccess) return pkv::cuda_error(e, "cudaStreamGetCaptureInfo");
  if (status != cudaStreamCaptureStatusActive) *id = 0;
  return PKV_OK;
}

}  // namespace

extern "C" {

pkv_status pkv_capture_id(void* stream, uint64_t* id) {
  pkv::set_last_error("");
  if (!id) {
    pkv::set_last_error("id is NULL");
    return PKV_ERR_INVALID_ARG;
  }
  unsigned long long x = 0;
  const pkv_status st = capture_info(stream, &x, nullptr);
  *id = x;
  return st;
}

pkv_status pkv_capture_watch(void* stream) {
  pkv::set_last_error("");
  unsigned long long id = 0;
  cudaGraph_t graph = nullptr;
  const pkv_status st = capture_info(stream, &id, &graph);
  if (st != PKV_OK) return st;
  if (id == 0) {
    pkv::set_last_error("the stream is not being captured");
    return PKV_ERR_INVALID_ARG;
  }
  Watch* w = nullptr;
  try {
    Gone& g = gone();
    std::lock_guard<std::mutex> lk(g.mu);
    g.ids.reserve(g.watched + 1);  // the destructor does not allocate
    w = new Watch{id};
    ++g.watched;
  } catch (const std::bad_alloc&) {
    pkv::set_last_error("out of host memory");
    return PKV_ERR_INVALID_ARG;
  }
  auto undo = [&]() {
    std::lock_guard<std::mutex> lk(gone().mu);
    --gone().watched;
  };
  cudaUserObject_t obj = nullptr;
  cudaError_t e = cudaUserObjectCreate(&obj, w, note, 1, cudaUserObjectNoDestructorSync);
  if (e != cudaSuccess) {
    delete w;
    undo();
    return pkv::cuda_error(e, "cudaUserObjectCreate");
  }
  e = cudaGraphRetainUserObject(graph, obj, 1, cudaGraphUserObjectMove);
  if (e != cudaSuccess) {
    cudaUserObjectRelease(obj, 1);  // notes the id: nothing holds it any longer
    return pkv::cuda_error(e, "cudaGraphRetainUserObject");
  }
  return PKV_OK;
}

pkv_status pkv_capture_gone(uint64_t* id) {
  pkv::set_last_error("");
  if (!id) {
    pkv::set_last_error("id is NULL");
    return PKV_ERR_INVALID_ARG;
  }
  std::lock_guard<std::mutex> lk(gone().mu);
  *id = 0;
  if (!gone().ids.empty()) {
    *id = gone().ids.back();
    gone().ids.pop_back();
    --gone().watched;
  }
  return PKV_OK;
}

}  // extern "C"
