// The opt-in launch profiler (muon_profile_begin / muon_profile_end): kinds of
// launches and the scope that brackets one launch with CUDA events.
#pragma once

#include <cuda_runtime.h>

#include <mutex>
#include <vector>

namespace muon {

enum ProfKind {
  kProfPack, kProfNorm, kProfSyrkTc, kProfGemmTc, kProfGemmSimt, kProfUnpack, kProfFusedSmall, kProfTf32, kProfChain,
  kProfStatus, kProfSplit, kProfExpertSort, kProfExpertGather, kProfExpertCombine, kProfExpertCombineBackward,
  kProfExpertProduct, kProfExpertSimt, kProfBlockChain, kProfKinds
};
struct ProfRec {
  int kind;
  cudaEvent_t a, b;
  double flops, exec_flops, bytes;
};
struct Profiler {
  bool on = false;
  std::vector<ProfRec> recs;
  std::mutex mu;
};
Profiler& profiler();  // the library's one profiler (api.cu)
// Brackets one launch with events on its stream while profiling is on.
struct ProfScope {
  ProfRec rec{};
  bool active = false;
  cudaStream_t s;
  ProfScope(int kind, double flops, double bytes, cudaStream_t st, double exec_flops = -1.0) : s(st) {
    Profiler& P = profiler();
    if (!P.on) return;
    rec.kind = kind; rec.flops = flops; rec.bytes = bytes;
    rec.exec_flops = exec_flops < 0.0 ? flops : exec_flops;
    if (cudaEventCreate(&rec.a) != cudaSuccess) return;
    if (cudaEventCreate(&rec.b) != cudaSuccess) { cudaEventDestroy(rec.a); return; }
    cudaEventRecord(rec.a, s);
    active = true;
  }
  ~ProfScope() {
    if (!active) return;
    cudaEventRecord(rec.b, s);
    Profiler& P = profiler();
    try {
      std::lock_guard<std::mutex> g(P.mu);
      P.recs.push_back(rec);
    } catch (...) {  // std::bad_alloc: the launch has gone out, it is not profiled
      cudaEventDestroy(rec.a);
      cudaEventDestroy(rec.b);
    }
  }
};

}  // namespace muon
