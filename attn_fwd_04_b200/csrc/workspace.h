// workspace.h -- which host thread may use a stream's workspace, and for how long.
//
// A call's launches hand results to one another through its stream's block (a
// decode's partial outputs and the merge that reads them), and a call that needs
// more frees the block and allocates another in the stream's order.  Both are right
// only if no other call of that stream is made in between: a call holds the block
// from its lookup to its last launch.  Calls on other streams are not waited for.
// (Host code without CUDA in it.)
#pragma once
#include <cstddef>
#include <memory>
#include <mutex>
#include <utility>
#include <vector>

namespace fa {

struct StreamBlock {
    void* stream = nullptr;
    void* ptr = nullptr;
    std::size_t bytes = 0;
    bool gone = false;  // released: nobody's any more
    std::mutex busy;
};

// A block in the hands of one call, until this is destroyed.
class WorkspaceHold {
  public:
    WorkspaceHold() = default;
    explicit WorkspaceHold(std::shared_ptr<StreamBlock> b) : block_(std::move(b)), lock_(block_->busy) {}
    StreamBlock* operator->() const { return block_.get(); }

  private:
    std::shared_ptr<StreamBlock> block_;  // (outlives the lock)
    std::unique_lock<std::mutex> lock_;
};

class StreamBlocks {
  public:
    // The stream's block, an empty one at first, once no other call has it.
    WorkspaceHold take(void* stream) {
        for (;;) {
            WorkspaceHold hold(find(stream));
            if (!hold->gone) return hold;
        }
    }

    // All blocks, none of them held, no longer anyone's: for the caller to free.
    std::vector<std::shared_ptr<StreamBlock>> clear() {
        std::vector<std::shared_ptr<StreamBlock>> out;
        {
            std::lock_guard<std::mutex> lock(mu_);
            all_.insert(all_.end(), unfreed_.begin(), unfreed_.end());
            unfreed_.clear();
            out.swap(all_);
        }
        for (auto& b : out) WorkspaceHold(b)->gone = true;
        return out;
    }

    // One of those that could not be freed: the next clear gives it again.
    void keep(std::shared_ptr<StreamBlock> b) {
        std::lock_guard<std::mutex> lock(mu_);
        unfreed_.push_back(std::move(b));
    }

  private:
    std::shared_ptr<StreamBlock> find(void* stream) {
        std::lock_guard<std::mutex> lock(mu_);
        for (auto& b : all_)
            if (b->stream == stream) return b;
        auto b = std::make_shared<StreamBlock>();
        b->stream = stream;
        all_.push_back(b);
        return b;
    }

    std::mutex mu_;
    std::vector<std::shared_ptr<StreamBlock>> all_, unfreed_;
};

}  // namespace fa
