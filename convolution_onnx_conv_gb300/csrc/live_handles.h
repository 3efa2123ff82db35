// The count of handles and layers in existence (conv_fused_debug_live_handles), kept by api.cu.
#pragma once

namespace convf {

// A member of every handle and layer.
struct LiveHandleCount {
  LiveHandleCount();
  LiveHandleCount(const LiveHandleCount&);
  LiveHandleCount& operator=(const LiveHandleCount&) = default;
  ~LiveHandleCount();
};

}  // namespace convf
